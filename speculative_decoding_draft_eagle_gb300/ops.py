"""Python binding of the C ABI, with the same names: argument marshalling only.

Every computation runs in the CUDA library; torch supplies device memory,
streams and output allocation.  Functions take torch CUDA tensors and enqueue
on the current torch stream (or ``stream=``, which the caller orders after what
its inputs come from, and before what reads its results).  None of them records
an autograd graph, whatever its arguments require; ``ttt.ttt_attention`` does.
"""

from __future__ import annotations

import ctypes
import math
import struct
import threading
from typing import List, Optional, Sequence, Tuple

import torch

from ._lib import check, lib

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
    "stt_top_logits",
    "soft_ce_topk_fwd_bwd",
    "stt_sample",
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


def _on(stream, call, *args, held=()):
    """`call` with `stream` (a torch stream or a handle) current: what it allocates belongs
    to that stream.  Memory of the caller's stream may still be in use by work that was
    queued there before; the other stream would write it without waiting for that.  The
    caller's stream is recorded on the results, which it goes on to use, and `stream` on
    what the caller gave to be written (the results, `held`)."""
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    here = torch.cuda.current_stream()
    if stream == here:
        return call(*args)
    with torch.cuda.stream(stream):
        result = call(*args)
    for r in (*(result if isinstance(result, tuple) else (result,)), *held):
        for t in r if isinstance(r, (list, tuple)) else (r,):
            if t is not None:
                t.record_stream(stream)
                t.record_stream(here)
    return result


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
    if stream is not None:
        return _on(stream, stt_attn_fwd, q, k_blocks, v_blocks, T, scale, out, lse)
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
    if stream is not None:
        return _on(stream, stt_attn_bwd, q, k_blocks, v_blocks, T, out, dout, lse, scale,
                   dq, dk_blocks, dv_blocks, workspace, held=(workspace,))
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
    if stream is not None:
        return _on(stream, stt_attn_bwd_ex, q, k_blocks, v_blocks, T, out, dout, lse, dq,
                   dk_blocks, dv_blocks, scale, accumulate, workspace, held=(workspace,))
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
    if stream is not None:
        return _on(stream, soft_ce_fwd_bwd_inplace, z, p, g, row_loss, loss, workspace,
                   want_row_loss, held=(z, workspace))
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
    if stream is not None:
        return _on(stream, soft_ce_fwd_bwd_inplace_ex, z, p, g, row_loss, loss, workspace,
                   held=(z, workspace))
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
    if stream is not None:
        return _on(stream, soft_ce_fwd_bwd_inplace_noalloc, z, p, g, row_loss, loss,
                   held=(z,))
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
    if stream is not None:
        return _on(stream, stt_lm_head_ce, h, W, p, g, dh, dW, row_loss, loss, workspace,
                   held=(workspace,))
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
    if stream is not None:
        return _on(stream, stt_verify, p_target, p_draft, draft_tokens, u_accept, u_sample,
                   n_accepted, out_tokens)
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


# The operators around the paged cache are called once per layer and token, so
# their checks take one short path for a good argument and explain only a bad one.
# The structs of the C ABI are packed as bytes.
_ROPE = struct.Struct("@PPPiIff")
_PAGES = struct.Struct("@PPPPPqqqiiiiii")
_LOGITS = struct.Struct("@PPPPPPPPPPiii")


def _current():
    """The current device, and its current stream's handle."""
    dev = torch.cuda.current_device()
    return dev, torch._C._cuda_getCurrentRawStream(dev)


def _refuse(t, name, dtype, shape, dev):
    """Raises what is wrong with a tensor argument."""
    _need(t, name, dtype, shape)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    raise ValueError(f"{name} is not a usable tensor")


def _arg(t, name, dtype, shape, dev) -> int:
    """Address of a contiguous tensor of that type and shape on the current device."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == dev
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, dev)


def _rows(t, name, shape, dev):
    """Address of bf16 rows (the last dimension) that are dense but for the distance
    between them, and that distance."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    width = shape[-1]
    if t.get_device() != dev or t.dtype is not torch.bfloat16 or t.shape != shape:
        if t.dtype is not torch.bfloat16:
            raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    if t.is_contiguous():
        return t.data_ptr(), width
    stride = t.stride()
    three = len(shape) == 3 and shape[0] > 1
    ld = stride[-2] if shape[-2] > 1 else (stride[0] if three else width)
    if ((width > 1 and stride[-1] != 1) or ld < width or
            (three and stride[0] != shape[1] * ld)):
        raise ValueError(f"{name} must be dense apart from the distance between its rows")
    return t.data_ptr(), ld


def _new(shape, dtype, dev):
    return torch.empty(shape, device=dev, dtype=dtype)


_scratch_of = threading.local()


def _scratch(n: int, dev: int, raw: int) -> torch.Tensor:
    """A workspace of n bytes for one call.  Eager calls of a thread on one stream
    follow one another there and share one, kept from call to call; a call that is
    captured has its own."""
    if torch._C._cuda_isCurrentStreamCapturing():
        return _new((n,), torch.uint8, dev)
    kept = _scratch_of.__dict__
    t = kept.get((dev, raw))
    if t is None or t.numel() < n:
        t = kept[dev, raw] = _new((n,), torch.uint8, dev)
    return t


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


STT_ROPE_INTERLEAVED = 0x1
STT_ROPE_BF16_GRADS = 0x2


def _rope(freq, w_q, w_k, D, eps, interleaved, amplitude, dev) -> bytes:
    R, f = 0, 0
    if freq is not None:
        if not isinstance(freq, torch.Tensor) or freq.dim() != 1:
            raise ValueError("freq must be [R/2]")
        f = _arg(freq, "freq", torch.float64, freq.shape, dev)
        R = 2 * freq.numel()
    return _ROPE.pack(
        f if R else 0, 0 if w_q is None else _arg(w_q, "w_q", torch.bfloat16, (D,), dev),
        0 if w_k is None else _arg(w_k, "w_k", torch.bfloat16, (D,), dev), R,
        STT_ROPE_INTERLEAVED if interleaved else 0, amplitude, eps)


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
    if stream is not None:
        return _on(stream, stt_qkv_rope_fwd, qkv, H, H_kv, D, positions, freq, w_q, w_k, eps,
                   interleaved, amplitude, q, k, v)
    dev, raw = _current()
    if qkv.dim() != 3:
        raise ValueError("qkv must be [B, S, (H + 2 H_kv) D]")
    B, S, _ = qkv.shape
    x, ld = _rows(qkv, "qkv", (B, S, (H + 2 * H_kv) * D), dev)
    rope = _rope(freq, w_q, w_k, D, eps, interleaved, amplitude, dev)
    bf16 = torch.bfloat16
    if q is None:
        q = _new((B, H, S, D), bf16, dev)
    if k is None:
        k = _new((B, H_kv, S, D), bf16, dev)
    if v is None:
        v = _new((B, H_kv, S, D), bf16, dev)
    st = lib().stt_qkv_rope_fwd(
        x, ld, None if positions is None else _arg(positions, "positions", torch.int32, (B, S), dev),
        B, S, H, H_kv, D, rope, _arg(q, "q", bf16, (B, H, S, D), dev),
        _arg(k, "k", bf16, (B, H_kv, S, D), dev), _arg(v, "v", bf16, (B, H_kv, S, D), dev), raw)
    if st:
        check("stt_qkv_rope_fwd", st)
    return q, k, v


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
    if stream is not None:
        return _on(stream, stt_qkv_rope_bwd, dq, dk, dv, qkv, positions, freq, w_q, w_k, eps,
                   interleaved, amplitude, dqkv, dw_q, dw_k, workspace, held=(workspace,))
    dev, raw = _current()
    if dq.dim() != 4 or dk.dim() != 4:
        raise ValueError("dq must be [B, H, S, D] and dk, dv [B, H_kv, S, D]")
    B, H, S, D = dq.shape
    H_kv = dk.shape[1]
    t = dq.dtype
    if t is not torch.float32 and t is not torch.bfloat16:
        raise ValueError("dq must be float32 or bfloat16")
    C = (H + 2 * H_kv) * D
    p_dq = _arg(dq, "dq", t, (B, H, S, D), dev)
    p_dk = _arg(dk, "dk", t, (B, H_kv, S, D), dev)
    p_dv = _arg(dv, "dv", t, (B, H_kv, S, D), dev)
    rope = _rope(freq, w_q, w_k, D, eps, interleaved, amplitude, dev)
    norm = w_q is not None or w_k is not None
    x, ld = None, C
    if norm:
        if qkv is None:
            raise ValueError("qkv is needed for the gradient of the norm")
        x, ld = _rows(qkv, "qkv", (B, S, C), dev)
    if dqkv is None:
        dqkv = _new((B, S, C), torch.bfloat16, dev)
    p_d, ld_d = _rows(dqkv, "dqkv", (B, S, C), dev)
    p_wq = p_wk = p_ws = None
    n_ws = 0
    if (dw_q is not None and w_q is None) or (dw_k is not None and w_k is None):
        raise ValueError("a weight's gradient is asked for without the weight")
    if w_q is not None:
        if dw_q is None:
            dw_q = _new((D,), torch.float32, dev)
        p_wq = _arg(dw_q, "dw_q", torch.float32, (D,), dev)
    if w_k is not None:
        if dw_k is None:
            dw_k = _new((D,), torch.float32, dev)
        p_wk = _arg(dw_k, "dw_k", torch.float32, (D,), dev)
    if norm:
        if workspace is None:
            n_ws = lib().stt_qkv_rope_bwd_workspace_size(D)
            workspace = _scratch(n_ws, dev, raw)
            p_ws = workspace.data_ptr()
        else:
            p_ws = _arg(workspace, "workspace", workspace.dtype, workspace.shape, dev)
            n_ws = workspace.numel() * workspace.element_size()
    st = lib().stt_qkv_rope_bwd(
        p_dq, p_dk, p_dv, x, ld,
        None if positions is None else _arg(positions, "positions", torch.int32, (B, S), dev),
        B, S, H, H_kv, D, rope, STT_ROPE_BF16_GRADS if t is torch.bfloat16 else 0, p_d, ld_d, p_wq,
        p_wk, p_ws, n_ws, raw)
    if st:
        check("stt_qkv_rope_bwd", st)
    return dqkv, dw_q, dw_k


def _pages(k_cache, v_cache, cu_q, seq_lens, page_table, dev):
    """The packed stt_pages, and H_kv, D and B."""
    bf16 = torch.bfloat16
    if (k_cache.dtype is not bf16 or v_cache.dtype is not bf16 or k_cache.dim() != 4
            or k_cache.get_device() != dev or v_cache.get_device() != dev):
        raise ValueError("k_cache and v_cache must be bfloat16 [num_pages, H_kv, page_size, D] "
                         f"on cuda:{dev}")
    stride = k_cache.stride()
    n, H_kv, page, D = shape = k_cache.shape
    if v_cache.shape != shape or v_cache.stride() != stride:
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    if stride[3] != 1 and D > 1 and k_cache.numel():
        raise ValueError("the elements of a cached head must be contiguous")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    B, max_pages = page_table.shape
    if n == 1 or H_kv == 1 or page == 1:  # a dimension of one element has no stride of its own
        stride = [s if size > 1 else max(8, (D + 7) // 8 * 8) for s, size in zip(stride, shape)]
    return _PAGES.pack(
        k_cache.data_ptr(), v_cache.data_ptr(),
        _arg(page_table, "page_table", torch.int32, (B, max_pages), dev),
        _arg(cu_q, "cu_q", torch.int32, (B + 1,), dev),
        _arg(seq_lens, "seq_lens", torch.int32, (B,), dev), stride[0], stride[1], stride[2], B,
        H_kv, D, page, n, max_pages), H_kv, D, B


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
    if stream is not None:
        return _on(stream, stt_kv_append, qkv, H, k_cache, v_cache, cu_q, seq_lens, page_table,
                   positions, freq, w_q, w_k, eps, interleaved, amplitude, q)
    dev, raw = _current()
    pages, H_kv, D, _ = _pages(k_cache, v_cache, cu_q, seq_lens, page_table, dev)
    if qkv.dim() != 2:
        raise ValueError("qkv must be [N, (H + 2 H_kv) D]")
    N = qkv.shape[0]
    x, ld = _rows(qkv, "qkv", (N, (H + 2 * H_kv) * D), dev)
    rope = _rope(freq, w_q, w_k, D, eps, interleaved, amplitude, dev)
    if q is None:
        q = _new((N, H, D), torch.bfloat16, dev)
    st = lib().stt_kv_append(
        x, ld, None if positions is None else _arg(positions, "positions", torch.int32, (N,), dev),
        N, H, pages, rope, _arg(q, "q", torch.bfloat16, (N, H, D), dev), raw)
    if st:
        check("stt_kv_append", st)
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
    left as they are.  out may not overlap q."""
    if stream is not None:
        return _on(stream, stt_paged_attn, q, k_cache, v_cache, cu_q, seq_lens, page_table,
                   scale, tree_mask, out, lse, workspace, held=(workspace,))
    dev, raw = _current()
    pages, H_kv, D, B = _pages(k_cache, v_cache, cu_q, seq_lens, page_table, dev)
    if q.dim() != 3 or q.shape[2] != D or q.dtype is not torch.bfloat16 or q.get_device() != dev:
        raise ValueError(f"q must be bfloat16 [N, H, {D}] on cuda:{dev}")
    N, H, _ = q.shape
    ld = H * D
    if not q.is_contiguous():
        s = q.stride()
        if s[2] != 1 or (H > 1 and s[1] != D) or (N > 1 and s[0] < ld):
            raise ValueError("q must be dense apart from the distance between its rows")
        if N > 1:
            ld = s[0]
    words, tree = 0, None
    if tree_mask is not None:
        if tree_mask.dim() != 2 or (N > 0 and tree_mask.shape[1] == 0):
            raise ValueError("tree_mask must be [N, words], at least one word")
        words = tree_mask.shape[1]
        tree = _arg(tree_mask, "tree_mask", torch.int32, (N, words), dev)
    if out is None:
        out = _new((N, H, D), torch.bfloat16, dev)
    if lse is None:
        lse = _new((N, H), torch.float32, dev)
    L = lib()
    if workspace is None:
        n_ws = L.stt_paged_attn_workspace_size(N, B, H, H_kv, D)
        workspace = _scratch(n_ws, dev, raw)
        p_ws = workspace.data_ptr()
    else:
        p_ws = _arg(workspace, "workspace", workspace.dtype, workspace.shape, dev)
        n_ws = workspace.numel() * workspace.element_size()
    st = L.stt_paged_attn(
        q.data_ptr(), ld, N, H, pages, D ** -0.5 if scale is None else scale, tree, words,
        _arg(out, "out", torch.bfloat16, (N, H, D), dev),
        _arg(lse, "lse", torch.float32, (N, H), dev), p_ws, n_ws, raw)
    if st:
        check("stt_paged_attn", st)
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
    draft_tokens int32 [B, >= rows - 1] (a chain: in a tree of drafts a position would
    need its ancestors, and each path goes as a sequence of its own).  bias fp32 [V], [1, V] or [B, V]; mask int32
    [N, ceil(V / 32)], bit v % 32 of word v / 32 set where v is allowed.  out may be z
    itself where that is fp32."""
    if stream is not None:
        return _on(stream, stt_logits_process, z, rows, temperature, repetition, frequency,
                   presence, tokens, cu_tokens, n_prompt, draft_tokens, bias, mask, raw, out)
    dev, on = _current()
    if z.dim() != 2:
        raise ValueError("z must be [N, V]")
    N, V = z.shape
    t, i32, f32 = z.dtype, torch.int32, torch.float32
    if t is not f32 and t is not torch.bfloat16:
        raise ValueError("z must be float32 or bfloat16")
    p_z = _arg(z, "z", t, (N, V), dev)
    if rows < 1 or N % rows:
        raise ValueError("rows must be positive and divide N")
    B = N // rows
    of = (B,)
    p_t = 0 if temperature is None else _arg(temperature, "temperature", f32, of, dev)
    p_r = 0 if repetition is None else _arg(repetition, "repetition", f32, of, dev)
    p_f = 0 if frequency is None else _arg(frequency, "frequency", f32, of, dev)
    p_p = 0 if presence is None else _arg(presence, "presence", f32, of, dev)
    if (tokens is None) != (cu_tokens is None):
        raise ValueError("tokens and cu_tokens go together")
    p_tok = p_cu = p_np = p_dr = p_b = p_m = n_tok = draft_ld = bias_rows = 0
    if tokens is not None:
        if tokens.dim() != 1:
            raise ValueError("tokens must be [total]")
        p_tok = _arg(tokens, "tokens", i32, tokens.shape, dev)
        p_cu = _arg(cu_tokens, "cu_tokens", i32, (B + 1,), dev)
    if n_prompt is not None:
        if tokens is None:
            raise ValueError("n_prompt is given without tokens")
        p_np = _arg(n_prompt, "n_prompt", i32, of, dev)
    if tokens is not None:
        n_tok = tokens.numel()
        if n_tok == 0:  # an empty history has no address
            p_tok = p_cu = p_np = 0
    if draft_tokens is not None:
        if draft_tokens.dim() != 2 or draft_tokens.shape[1] < rows - 1:
            raise ValueError(f"draft_tokens must be [B, at least {rows - 1}]")
        draft_ld = draft_tokens.shape[1]
        p_dr = _arg(draft_tokens, "draft_tokens", i32, (B, draft_ld), dev) if draft_ld else 0
    if bias is not None:
        bias_rows = 1 if bias.dim() == 1 else bias.shape[0]
        if bias_rows != 1 and bias_rows != B:
            raise ValueError("bias must be [V], [1, V] or [B, V]")
        p_b = _arg(bias, "bias", f32, (V,) if bias.dim() == 1 else (bias_rows, V), dev)
    if mask is not None:
        p_m = _arg(mask, "mask", i32, (N, (V + 31) // 32), dev)
    if out is None:
        out = _new((N, V), f32, dev)
    params = _LOGITS.pack(p_t, p_r, p_f, p_p, p_tok, p_cu, p_np, p_dr, p_b, p_m, n_tok,
                          draft_ld, bias_rows)
    st = lib().stt_logits_process(
        p_z, N, V, rows, params,
        (STT_LOGITS_BF16 if t is torch.bfloat16 else 0) | (STT_LOGITS_RAW if raw else 0),
        _arg(out, "out", f32, (N, V), dev), on)
    if st:
        check("stt_logits_process", st)
    return out


def _logits(z, name, dev, dtype=None, shape=None):
    """Address of rows of logits [N, V] (fp32 or bf16, or `dtype`) that are dense but for
    the distance between them, and that distance."""
    if not isinstance(z, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if z.dim() != 2 or (shape is not None and z.shape != shape):
        raise ValueError(f"{name} must be [N, V]" if shape is None else
                         f"{name} must have shape {tuple(shape)}, got {tuple(z.shape)}")
    t = z.dtype
    if t is not dtype if dtype is not None else (t is not torch.float32 and t is not torch.bfloat16):
        raise ValueError(f"{name} must be {dtype or 'float32 or bfloat16'}, got {t}")
    if z.get_device() != dev:
        raise ValueError(f"{name} is on {z.device}, the current device is cuda:{dev}")
    N, V = z.shape
    if z.is_contiguous():
        return z.data_ptr(), V
    ld, one = z.stride()
    if (V > 1 and one != 1) or (N > 1 and ld < V):
        raise ValueError(f"{name} must be dense apart from the distance between its rows")
    return z.data_ptr(), ld if N > 1 else V


def _apart(a, ld_a, b, ld_b, name):
    """Refuses rows b [N, V] that share memory with the rows a, unless they are a."""
    N, V = a.shape
    pa, pb, sa, sb = a.data_ptr(), b.data_ptr(), a.element_size(), b.element_size()
    if N == 0 or (pa == pb and sa == sb and (ld_a == ld_b or N == 1)):
        return
    if pa >= pb + ((N - 1) * ld_b + V) * sb or pb >= pa + ((N - 1) * ld_a + V) * sa:
        return
    if ld_a * sa == ld_b * sb:  # columns of one wider buffer
        off = (pb - pa) % (ld_a * sa)
        if off >= V * sa and off + V * sb <= ld_a * sa:
            return
    raise ValueError(f"{name} overlaps the logits")


def stt_top_logits(z: torch.Tensor, K: int, temperature: float = 1.0,
                   values: Optional[torch.Tensor] = None, indices: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, stream=None
                   ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The K largest logits of every row of z [N, V] (fp32 or bf16; rows may be a slice of
    wider ones), the largest first and the lower index first among equals, -inf never.

    Returns (values fp32 [N, K], -inf past the row's last; indices int32 [N, K], -1 there;
    lse fp32 [N] = log sum_v exp(z_v / temperature)): what soft_ce_topk_fwd_bwd takes of a
    teacher, or a draft tree's candidates, whose log-probability is
    values / temperature - lse."""
    if stream is not None:
        return _on(stream, stt_top_logits, z, K, temperature, values, indices, lse)
    dev, raw = _current()
    p_z, ld = _logits(z, "z", dev)
    N, V = z.shape
    if not 1 <= K <= V:
        raise ValueError(f"K must be 1..{V}, got {K}")
    f32, i32 = torch.float32, torch.int32
    if values is None:
        values = _new((N, K), f32, dev)
    if indices is None:
        indices = _new((N, K), i32, dev)
    if lse is None:
        lse = _new((N,), f32, dev)
    st = lib().stt_top_logits(
        p_z, ld, N, V, K, temperature, STT_LOGITS_BF16 if z.dtype is torch.bfloat16 else 0,
        _arg(values, "values", f32, (N, K), dev), _arg(indices, "indices", i32, (N, K), dev),
        _arg(lse, "lse", f32, (N,), dev), raw)
    if st:
        check("stt_top_logits", st)
    return values, indices, lse


def soft_ce_topk_fwd_bwd(z: torch.Tensor, t_values: torch.Tensor, t_indices: torch.Tensor,
                         g: torch.Tensor, t_lse: Optional[torch.Tensor] = None,
                         temperature: float = 1.0, dz: Optional[torch.Tensor] = None,
                         row_loss: Optional[torch.Tensor] = None,
                         loss: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None):
    """Soft-CE of logits z [N, V] (fp32 or bf16; rows may be a slice of wider ones) against a
    teacher's top logits t_values fp32 and t_indices int32 [N, K] (an index outside [0, V),
    such as -1, is no entry), with the gradient.

    Both sides are divided by `temperature`.  With t_lse fp32 [N], the teacher's
    log-sum-exp at it (stt_top_logits), the targets are the teacher's probabilities;
    without, they are renormalised over the entries.  g fp32 [N]: upstream gradient of each
    row's loss, 0 for a masked row.  The gradient goes over z, or into dz (z's type).
    Returns (loss [1] = sum g row_loss, row_loss [N], the gradient)."""
    if stream is not None:
        return _on(stream, soft_ce_topk_fwd_bwd, z, t_values, t_indices, g, t_lse, temperature,
                   dz, row_loss, loss, workspace, held=(workspace,))
    dev, raw = _current()
    p_z, ld = _logits(z, "z", dev)
    N, V = z.shape
    f32 = torch.float32
    if t_values.dim() != 2 or t_values.shape[1] < 1:
        raise ValueError("t_values must be [N, K], K at least 1")
    K = t_values.shape[1]
    p_v = _arg(t_values, "t_values", f32, (N, K), dev)
    p_i = _arg(t_indices, "t_indices", torch.int32, (N, K), dev)
    p_g = _arg(g, "g", f32, (N,), dev)
    p_l = None if t_lse is None else _arg(t_lse, "t_lse", f32, (N,), dev)
    if dz is None:
        dz = z
    p_d, ld_d = _logits(dz, "dz", dev, z.dtype, z.shape)
    if dz is not z:
        _apart(z, ld, dz, ld_d, "dz")
    if row_loss is None:
        row_loss = _new((N,), f32, dev)
    if loss is None:
        loss = _new((1,), f32, dev)
    L = lib()
    if workspace is None:
        n_ws = L.soft_ce_workspace_size(N, V)
        workspace = _scratch(n_ws, dev, raw)
        p_ws = workspace.data_ptr()
    else:
        p_ws = _arg(workspace, "workspace", workspace.dtype, workspace.shape, dev)
        n_ws = workspace.numel() * workspace.element_size()
    st = L.soft_ce_topk_fwd_bwd(
        p_z, ld, p_v, p_i, p_l, p_g, N, V, K, temperature,
        STT_CE_BF16 if z.dtype is torch.bfloat16 else 0, p_d, ld_d,
        _arg(row_loss, "row_loss", f32, (N,), dev), _arg(loss, "loss", f32, (1,), dev), p_ws, n_ws,
        raw)
    if st:
        check("soft_ce_topk_fwd_bwd", st)
    return loss, row_loss, dz


def stt_sample(z: torch.Tensor, u: Optional[torch.Tensor] = None, rows: int = 1,
               temperature: Optional[torch.Tensor] = None, top_k: Optional[torch.Tensor] = None,
               top_p: Optional[torch.Tensor] = None, min_p: Optional[torch.Tensor] = None,
               probs: Optional[torch.Tensor] = None, want_probs: bool = False,
               tokens: Optional[torch.Tensor] = None, logprobs: Optional[torch.Tensor] = None,
               stream=None):
    """Logits z [N, V] (fp32 or bf16; rows may be a slice of wider ones; `rows` consecutive
    ones for each of the B = N / rows sequences) to the distribution that a sequence's
    temperature (0: greedy), top_k (int32, <= 0: off), top_p and min_p (fp32), each [B] or
    None, leave, and with u fp32 [N] in [0, 1) a token drawn from it.

    Kept are the top_k largest logits (the lower index first among equals), of those the
    fewest that hold top_p of their probability, of those the ones min_p times as probable
    as the first.  The token is the smallest whose cumulated probability exceeds u.
    Returns (tokens int32 [N], logprobs fp32 [N], probs fp32 [N, V]); without u the first
    two are None, and probs is None unless it or want_probs is given, or u is not.  probs
    may be z itself where that is fp32."""
    if stream is not None:
        return _on(stream, stt_sample, z, u, rows, temperature, top_k, top_p, min_p, probs,
                   want_probs, tokens, logprobs)
    dev, raw = _current()
    p_z, ld = _logits(z, "z", dev)
    N, V = z.shape
    if rows < 1 or N % rows:
        raise ValueError("rows must be positive and divide N")
    f32, i32, of = torch.float32, torch.int32, (N // rows,)
    p_t = None if temperature is None else _arg(temperature, "temperature", f32, of, dev)
    p_k = None if top_k is None else _arg(top_k, "top_k", i32, of, dev)
    p_p = None if top_p is None else _arg(top_p, "top_p", f32, of, dev)
    p_m = None if min_p is None else _arg(min_p, "min_p", f32, of, dev)
    p_u = p_tok = p_log = p_pr = None
    ld_p = V
    if u is not None:
        p_u = _arg(u, "u", f32, (N,), dev)
        if tokens is None:
            tokens = _new((N,), i32, dev)
        if logprobs is None:
            logprobs = _new((N,), f32, dev)
        p_tok = _arg(tokens, "tokens", i32, (N,), dev)
        p_log = _arg(logprobs, "logprobs", f32, (N,), dev)
    elif tokens is not None or logprobs is not None:
        raise ValueError("tokens and logprobs are given without u")
    if probs is None and (want_probs or u is None):
        probs = _new((N, V), f32, dev)
    if probs is not None:
        p_pr, ld_p = _logits(probs, "probs", dev, f32, z.shape)
        if probs is not z:
            _apart(z, ld, probs, ld_p, "probs")
    st = lib().stt_sample(p_z, ld, N, V, rows, p_t, p_k, p_p, p_m, p_u,
                          STT_LOGITS_BF16 if z.dtype is torch.bfloat16 else 0, p_tok, p_log, p_pr,
                          ld_p, raw)
    if st:
        check("stt_sample", st)
    return tokens, logprobs, probs


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

"""Exact attention for GB300 (sm_103a).

``fwd(q, k, v, causal)`` returns ``(o, lse)`` for contiguous bf16 CUDA tensors of shape
[B, H, T, d] (d = 64 or 128): o = softmax(scale·QKᵀ [+causal mask])·V in bf16 and the
per-row natural-log logsumexp in fp32. ``fwd_kv`` attends Tq queries to Tk ≥ Tq keys
(bottom-right causal; key range split over CTAs when that fills the GPU), and
``fwd_block_sparse`` skips 128×128 blocks switched off by a block mask.
``bwd(q, k, v, o, lse, do, causal)`` returns the gradients (dq, dk, dv) (d = 64 or 128).
``fwd_mod`` and ``bwd_mod`` are attention with modified scores (a tanh cap, a bias by distance,
documents and prefixes through ``visible``, key heads shared by query heads) and its gradients;
``rope`` and ``rope_append`` turn queries and keys by their positions, and ``fwd_tree`` attends
new tokens (one, a chain, a tree of drafts) to a cache of ragged contexts.
The work is done by the CUDA kernels of ``libfa.so`` through its C ABI (include/fa.h);
this module only allocates outputs and workspace with PyTorch and passes pointers and the
current stream.
"""

from __future__ import annotations

import math

from ._binding import (  # noqa: F401
    EXPORTS,
    FA_ERR_INVALID_ARG,
    FA_ERR_LAUNCH,
    FA_ERR_MISALIGNED,
    FA_ERR_TIMEOUT,
    FA_ERR_UNSUPPORTED_DEVICE,
    FA_FLAG_TEST_STARVE_Q,
    FA_FLAG_TEST_STARVE_LATER_Q,
    FA_FLAG_CTA_PAIR,
    FA_OK,
    FAError,
    fa_bwd,
    fa_bwd_ex,
    fa_bwd_mod,
    fa_bwd_workspace_size,
    fa_fwd,
    fa_fwd_block_sparse,
    fa_fwd_ex,
    fa_fwd_fp8,
    fa_fwd_host,
    fa_fwd_host_workspace_size,
    fa_fwd_kv,
    fa_fwd_kv_workspace_size,
    fa_fwd_mod,
    fa_fwd_tree,
    fa_fwd_tree_workspace_size,
    fa_rope,
    fa_rope_append,
    fa_visible,
    fa_visible_size,
    lib,
    strerror,
    version,
)


def _check(t, name):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16")
    if t.dim() != 4 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [B, H, T, d] tensor")


def fwd(q, k, v, causal: bool = True, scale: float | None = None, out=None, lse=None,
        status=None, timeout_ns: int = 0, flags: int = 0):
    """Attention forward through libfa.so on the current CUDA stream.

    Returns (o, lse). ``out``/``lse`` may be given to reuse buffers. ``status``, an
    optional int32 CUDA tensor of one element, receives FA_ERR_TIMEOUT if an internal
    wait of the kernel ever gives up; ``timeout_ns`` bounds those waits (0: 2 s).
    ``flags`` is 0 except in tests of that path: FA_FLAG_TEST_STARVE_Q withholds every
    query-tile load, FA_FLAG_TEST_STARVE_LATER_Q those after each CTA's first unit; and
    FA_FLAG_CTA_PAIR (d = 64) runs the forward on CTA pairs sharing each tensor-core product
    (same results, slower on GB300 than the default).
    """
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
    if q.shape != k.shape or q.shape != v.shape:
        raise ValueError("q, k and v must have the same shape")
    B, H, T, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check(out, "out")
    if lse is None:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    stream = torch.cuda.current_stream(q.device).cuda_stream
    st_ptr = None if status is None else status.data_ptr()
    with torch.cuda.device(q.device):
        rc = fa_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                       lse.data_ptr(), B, H, T, d, causal, scale, st_ptr, timeout_ns, flags,
                       stream)
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd")
    return out, lse


def fwd_host(q, k, v, causal: bool = True, scale: float | None = None, out=None, lse=None,
             heads_per_chunk: int = 0, workspace=None, device=None, synchronize: bool = True):
    """Forward over host tensors (CPU bf16 [B, H, T, d], contiguous; page-locked for
    overlapped copies) through fa_fwd_host on ``device``'s current stream. Outputs are host
    tensors (page-locked when not given). With ``synchronize`` the stream is synchronised
    before returning; otherwise the caller must do so before reading them."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.is_cuda or t.dtype != torch.bfloat16 \
                or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous host bf16 [B, H, T, d] tensor")
    if q.shape != k.shape or q.shape != v.shape:
        raise ValueError("q, k and v must have the same shape")
    B, H, T, d = q.shape
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None \
        else torch.device(device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, pin_memory=True)
    if lse is None:
        lse = torch.empty((B, H, T), dtype=torch.float32, pin_memory=True)
    with torch.cuda.device(dev):
        if workspace is None:
            need = fa_fwd_host_workspace_size(B, H, T, d, heads_per_chunk)
            if need == 0:
                raise FAError(FA_ERR_INVALID_ARG, "fa_fwd_host_workspace_size")
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        s = torch.cuda.current_stream(dev)
        rc = fa_fwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                         lse.data_ptr(), B, H, T, d, causal, scale, heads_per_chunk,
                         workspace.data_ptr(), workspace.numel(), s.cuda_stream)
        if rc != FA_OK:
            raise FAError(rc, "fa_fwd_host")
        if synchronize:
            s.synchronize()
    return out, lse


def fwd_fp8(q8, q_scale: float, k8, k_scale: float, v, causal: bool = True,
            scale: float | None = None, out=None, lse=None):
    """Forward with e4m3 query/key codes (CUDA uint8 tensors [B, H, T, d]) and their
    per-tensor scales, bf16 v, through fa_fwd_fp8. Returns (o, lse)."""
    import torch
    for t, n in ((q8, "q8"), (k8, "k8")):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.uint8 \
                or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous CUDA uint8 [B, H, T, d] tensor")
    _check(v, "v")
    if q8.shape != k8.shape or q8.shape != v.shape:
        raise ValueError("q8, k8 and v must have the same shape")
    B, H, T, d = v.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out = torch.empty_like(v) if out is None else out
    if lse is None:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=v.device)
    stream = torch.cuda.current_stream(v.device).cuda_stream
    with torch.cuda.device(v.device):
        rc = fa_fwd_fp8(q8.data_ptr(), k8.data_ptr(), v.data_ptr(), out.data_ptr(),
                        lse.data_ptr(), q_scale, k_scale, B, H, T, d, causal, scale, stream)
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_fp8")
    return out, lse


def fwd_kv(q, k, v, causal: bool = True, scale: float | None = None, n_splits: int = 0,
           out=None, lse=None, workspace=None):
    """Queries q [B, H, Tq, d] against keys/values k, v [B, H, Tk, d] through fa_fwd_kv.

    causal aligns bottom-right (query i sees key j iff j ≤ i + Tk − Tq; needs Tq ≤ Tk).
    n_splits = 0 lets the library choose how many key ranges to spread over CTAs; the
    workspace for the partial results is allocated here unless one is passed.
    Returns (o, lse); a row that sees no key has o = 0 and lse = −inf.
    """
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
    if k.shape != v.shape or q.shape[:2] != k.shape[:2] or q.shape[3] != k.shape[3]:
        raise ValueError("q must be [B, H, Tq, d] and k, v [B, H, Tk, d]")
    B, H, Tq, d = q.shape
    Tk = k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty((B, H, Tq), dtype=torch.float32, device=q.device)
    with torch.cuda.device(q.device):
        need = fa_fwd_kv_workspace_size(B, H, Tq, Tk, d, n_splits)
        if need == 0:
            raise FAError(FA_ERR_INVALID_ARG, "fa_fwd_kv_workspace_size")
        if workspace is None and need > 1:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        ws_ptr = None if workspace is None else workspace.data_ptr()
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        stream = torch.cuda.current_stream(q.device).cuda_stream
        rc = fa_fwd_kv(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                       B, H, Tq, Tk, d, causal, scale, n_splits, ws_ptr, ws_bytes, stream)
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_kv")
    return out, lse


def fwd_block_sparse(q, k, v, block_mask, causal: bool = False, scale: float | None = None,
                     out=None, lse=None):
    """Self-attention with 128×128 blocks switched off by ``block_mask`` (a CUDA uint8
    tensor [ceil(T/128), ceil(T/128)] shared by all heads, or [B·H, ...] per head;
    nonzero = compute), through fa_fwd_block_sparse. Returns (o, lse); a row that sees
    no key has o = 0 and lse = −inf."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
    if q.shape != k.shape or q.shape != v.shape:
        raise ValueError("q, k and v must have the same shape")
    B, H, T, d = q.shape
    nb = q_tiles(T)
    if (not isinstance(block_mask, torch.Tensor) or not block_mask.is_cuda
            or block_mask.dtype != torch.uint8 or not block_mask.is_contiguous()):
        raise ValueError("block_mask must be a contiguous CUDA uint8 tensor")
    if tuple(block_mask.shape[-2:]) != (nb, nb) or block_mask.dim() not in (2, 3):
        raise ValueError(f"block_mask must be [{nb}, {nb}] or [B*H, {nb}, {nb}]")
    mask_heads = 1 if block_mask.dim() == 2 else block_mask.shape[0]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    stream = torch.cuda.current_stream(q.device).cuda_stream
    with torch.cuda.device(q.device):
        rc = fa_fwd_block_sparse(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                 lse.data_ptr(), block_mask.data_ptr(), mask_heads, B, H, T, d,
                                 causal, scale, stream)
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_block_sparse")
    return out, lse


def bwd_workspace(B: int, H: int, T: int, d: int, device=None):
    """A uint8 CUDA tensor large enough to serve as fa_bwd's workspace (torch allocations
    are 256-byte aligned)."""
    import torch
    n = fa_bwd_workspace_size(B, H, T, d)
    if n == 0:
        raise FAError(FA_ERR_INVALID_ARG, "fa_bwd_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def bwd(q, k, v, o, lse, do, causal: bool = True, scale: float | None = None, dq=None,
        dk=None, dv=None, workspace=None, status=None, timeout_ns: int = 0, flags: int = 0):
    """Attention backward through libfa.so on the current CUDA stream.

    ``o`` and ``lse`` are the outputs of ``fwd`` for the same q, k, v, causal and scale;
    ``do`` is the gradient of the loss with respect to o. Returns (dq, dk, dv).
    ``workspace`` (see ``bwd_workspace``) may be passed to reuse it between calls.
    """
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (do, "do")):
        _check(t, n)
    if not (q.shape == k.shape == v.shape == o.shape == do.shape):
        raise ValueError("q, k, v, o and do must have the same shape")
    B, H, T, d = q.shape
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, T) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [B, H, T] tensor")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for t, n in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        _check(t, n)
    if workspace is None:
        workspace = bwd_workspace(B, H, T, d, device=q.device)
    stream = torch.cuda.current_stream(q.device).cuda_stream
    st_ptr = None if status is None else status.data_ptr()
    with torch.cuda.device(q.device):
        rc = fa_bwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                       lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                       workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                       B, H, T, d, causal, scale, st_ptr, timeout_ns, flags, stream)
    if rc != FA_OK:
        raise FAError(rc, "fa_bwd")
    return dq, dk, dv


def bwd_flops(B: int, H: int, T: int, d: int, causal: bool) -> float:
    """Algorithmic FLOPs of one backward: five T×T×d products (S, dP, dV, dK, dQ), i.e.
    2.5 × the forward's count, halved when causal."""
    return 2.5 * flops(B, H, T, d, causal)


def flops(B: int, H: int, T: int, d: int, causal: bool) -> float:
    """Algorithmic FLOPs of one forward: 4·B·H·T²·d (two T×T×d products), halved when
    causal (the convention the throughput figures are quoted in)."""
    f = 4.0 * B * H * T * T * d
    return f / 2.0 if causal else f


def hbm_bytes(B: int, H: int, T: int, d: int) -> float:
    """Algorithmic HBM bytes of one forward: read q, k, v once, write o (bf16) and lse (fp32)."""
    return B * H * T * (4.0 * d * 2 + 4.0)


def q_tiles(T: int, rows: int = 128) -> int:
    """Query-row tiles of ``rows`` rows covering a sequence of length T."""
    return -(-T // rows)


def _same_device(t, device, name):
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, as the other tensors")


def _check_int32(t, shapes, device, name):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or not t.is_contiguous() \
            or not t.is_cuda or tuple(t.shape) not in shapes:
        raise ValueError(f"{name} must be a contiguous CUDA int32 tensor of shape "
                         + " or ".join(str(list(s)) for s in shapes))
    _same_device(t, device, name)


class Visible:
    """Who sees whom in a batch, made by ``visible``: an opaque device buffer that ``fwd_mod`` and
    ``bwd_mod`` calls of the same B and T read."""

    __slots__ = ("buffer", "B", "T", "causal")

    def __init__(self, buffer, B: int, T: int, causal: bool):
        self.buffer, self.B, self.T, self.causal = buffer, B, T, causal


def visible(B: int, T: int, causal: bool = True, doc_ids=None, prefix_len=None, device=None,
            buffer=None) -> Visible:
    """The visibility of a batch of B sequences of T tokens, for every layer's ``fwd_mod`` and
    ``bwd_mod``.

    ``doc_ids`` (int32 [B, T]): a document is a maximal run of equal ids and sees itself only; a
    negative id is padding, which sees nothing and is seen by nothing. ``causal``: key j is
    visible to query i when j ≤ i or j is one of the first ``prefix_len`` tokens of their document
    (int32 [B], or [B, T] with each token holding its document's). ``buffer``, a uint8 CUDA tensor
    of fa_visible_size(B, T) bytes, may be given to reuse it.
    """
    import torch
    if device is None:
        device = next((t.device for t in (doc_ids, prefix_len, buffer) if t is not None),
                      torch.device("cuda", torch.cuda.current_device()))
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("the visibility lives on a CUDA device")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    if doc_ids is not None:
        _check_int32(doc_ids, ((B, T),), device, "doc_ids")
    if prefix_len is not None:
        _check_int32(prefix_len, ((B,), (B, T)), device, "prefix_len")
    need = fa_visible_size(B, T)
    if need == 0:
        raise FAError(FA_ERR_INVALID_ARG, "fa_visible_size")
    if buffer is None:
        buffer = torch.empty(need, dtype=torch.uint8, device=device)
    elif buffer.dtype != torch.uint8 or not buffer.is_contiguous():
        raise ValueError("buffer must be a contiguous uint8 CUDA tensor")
    _same_device(buffer, device, "buffer")
    with torch.cuda.device(device):
        rc = fa_visible(None if doc_ids is None else doc_ids.data_ptr(),
                        None if prefix_len is None else prefix_len.data_ptr(),
                        prefix_len is not None and prefix_len.dim() == 2, causal,
                        buffer.data_ptr(), buffer.numel(), B, T,
                        torch.cuda.current_stream(device).cuda_stream)
    if rc != FA_OK:
        raise FAError(rc, "fa_visible")
    return Visible(buffer, B, T, bool(causal))


def _check_slopes(slopes, H, device):
    import torch
    if slopes is None:
        return
    if not isinstance(slopes, torch.Tensor) or slopes.dtype != torch.float32 \
            or tuple(slopes.shape) != (H,) or not slopes.is_contiguous():
        raise ValueError(f"slopes must be a contiguous float32 tensor of shape [{H}]")
    _same_device(slopes, device, "slopes")


def _check_mod(q, k, v, seen, causal, slopes):
    """Shapes, devices and masks of a modified-score call; the causal flag that holds."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
        _same_device(t, q.device, n)
    B, H, T, d = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[2:] != q.shape[2:] \
            or H % max(1, k.shape[1]) != 0:
        raise ValueError("q must be [B, H, T, d] and k, v [B, Hkv, T, d] with Hkv a divisor of H")
    _check_slopes(slopes, H, q.device)
    if seen is None:
        return True if causal is None else bool(causal)
    if not isinstance(seen, Visible):
        raise TypeError("visible must be what visible() returned")
    if (seen.B, seen.T) != (B, T):
        raise ValueError(f"visible is for B {seen.B}, T {seen.T}, the tensors for B {B}, T {T}")
    if causal is not None and bool(causal) != seen.causal:
        raise ValueError("causal differs from what visible was made with")
    _same_device(seen.buffer, q.device, "visible")
    return seen.causal


def _check_lse(lse, shape, device):
    import torch
    if not isinstance(lse, torch.Tensor) or lse.dtype != torch.float32 \
            or tuple(lse.shape) != tuple(shape) or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 tensor of shape {list(shape)}")
    _same_device(lse, device, "lse")


def _check_like(t, ref, name):
    _check(t, name)
    _same_device(t, ref.device, name)
    if t.shape != ref.shape:
        raise ValueError(f"{name} must have shape {list(ref.shape)}")


def fwd_mod(q, k, v, visible=None, causal: bool | None = None, softcap: float = 0.0, slopes=None,
            scale: float | None = None, out=None, lse=None, status=None, timeout_ns: int = 0):
    """Attention with modified scores through fa_fwd_mod: z = scale·q·k, capped to
    softcap·tanh(z / softcap) when ``softcap`` > 0, lowered by slopes[h]·|i − j| when ``slopes``
    (float32 [H]) is given; softmax over the visible keys.

    q is [B, H, T, d], k and v [B, Hkv, T, d] with Hkv a divisor of H. ``visible`` (from
    ``visible()``) says who sees whom; without it ``causal`` does (None: causal). Returns
    (o, lse); a row that sees no key has o = 0 and lse = −inf.
    """
    import torch
    causal = _check_mod(q, k, v, visible, causal, slopes)
    B, H, T, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_like(out, q, "out")
    if lse is None:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    else:
        _check_lse(lse, (B, H, T), q.device)
    with torch.cuda.device(q.device):
        rc = fa_fwd_mod(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                        None if visible is None else visible.buffer.data_ptr(), causal, softcap,
                        None if slopes is None else slopes.data_ptr(), B, H, k.shape[1], T, d,
                        scale, None if status is None else status.data_ptr(), timeout_ns,
                        torch.cuda.current_stream(q.device).cuda_stream)
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_mod")
    return out, lse


def bwd_mod(q, k, v, o, lse, do, visible=None, causal: bool | None = None, softcap: float = 0.0,
            slopes=None, scale: float | None = None, dq=None, dk=None, dv=None, workspace=None,
            status=None, timeout_ns: int = 0):
    """Gradients of ``fwd_mod`` through fa_bwd_mod: (dq [B, H, T, d], dk, dv [B, Hkv, T, d]), from
    its outputs ``o`` and ``lse`` and the gradient ``do`` of o; the other arguments as there.
    ``workspace`` (see ``bwd_workspace``, with the query heads H) may be passed to reuse it."""
    import torch
    causal = _check_mod(q, k, v, visible, causal, slopes)
    for t, n in ((o, "o"), (do, "do")):
        _check_like(t, q, n)
    B, H, T, d = q.shape
    _check_lse(lse, (B, H, T), q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for t, r, n in ((dq, q, "dq"), (dk, k, "dk"), (dv, v, "dv")):
        _check_like(t, r, n)
    if workspace is None:
        workspace = bwd_workspace(B, H, T, d, device=q.device)
    _same_device(workspace, q.device, "workspace")
    with torch.cuda.device(q.device):
        rc = fa_bwd_mod(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                        lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                        workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                        None if visible is None else visible.buffer.data_ptr(), causal, softcap,
                        None if slopes is None else slopes.data_ptr(), B, H, k.shape[1], T, d,
                        scale, None if status is None else status.data_ptr(), timeout_ns,
                        torch.cuda.current_stream(q.device).cuda_stream)
    if rc != FA_OK:
        raise FAError(rc, "fa_bwd_mod")
    return dq, dk, dv


def fwd_tree_workspace(B: int, H: int, Hkv: int, Tq: int, Tmax: int, d: int, device=None):
    """A uint8 CUDA tensor large enough to serve as ``fwd_tree``'s workspace."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None \
        else torch.device(device)
    with torch.cuda.device(dev):
        n = fa_fwd_tree_workspace_size(B, H, Hkv, Tq, Tmax, d)
    if n == 0:
        raise FAError(FA_ERR_INVALID_ARG, "fa_fwd_tree_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=dev)


def fwd_tree(q, k_cache, v_cache, ctx_len, tree=None, depths=None, softcap: float = 0.0,
             slopes=None, scale: float | None = None, out=None, lse=None, workspace=None,
             status=None, timeout_ns: int = 0):
    """New tokens q [B, H, Tq, d] against caches [B, Hkv, Tmax, d] through fa_fwd_tree: sequence b
    holds ``ctx_len[b]`` tokens (int32 [B]; negative: inactive) and behind them, already written
    (``rope_append``), its Tq new ones.

    A new token sees the whole context and, of the new tokens, those where ``tree`` (uint8 or bool
    [Tq, Tq] or [B, Tq, Tq], nonzero = row t sees token s) says so; without it a chain: itself and
    the ones before. ``softcap`` and ``slopes`` as for ``fwd_mod``, the bias measured between
    positions ctx_len[b] + ``depths`` (int32 [Tq] or [B, Tq]; None: 0, 1, …). Returns (o, lse); a
    token that sees nothing has o = 0 and lse = −inf. ``workspace``: see ``fwd_tree_workspace``.
    """
    import torch
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _check(t, n)
        _same_device(t, q.device, n)
    B, H, Tq, d = q.shape
    Hkv, Tmax = k_cache.shape[1], k_cache.shape[2]
    if k_cache.shape != v_cache.shape or k_cache.shape[0] != B or k_cache.shape[3] != d \
            or H % max(1, Hkv) != 0:
        raise ValueError("q must be [B, H, Tq, d] and the caches [B, Hkv, Tmax, d] with Hkv a "
                         "divisor of H")
    _check_int32(ctx_len, ((B,),), q.device, "ctx_len")
    if tree is not None:
        if not isinstance(tree, torch.Tensor) or tree.dtype not in (torch.uint8, torch.bool) \
                or not tree.is_contiguous() or tuple(tree.shape) not in ((Tq, Tq), (B, Tq, Tq)):
            raise ValueError(f"tree must be a contiguous uint8 or bool tensor of shape "
                             f"[{Tq}, {Tq}] or [{B}, {Tq}, {Tq}]")
        _same_device(tree, q.device, "tree")
    if depths is not None:
        _check_int32(depths, ((Tq,), (B, Tq)), q.device, "depths")
    _check_slopes(slopes, H, q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_like(out, q, "out")
    if lse is None:
        lse = torch.empty((B, H, Tq), dtype=torch.float32, device=q.device)
    else:
        _check_lse(lse, (B, H, Tq), q.device)
    if workspace is None:
        workspace = fwd_tree_workspace(B, H, Hkv, Tq, Tmax, d, device=q.device)
    _same_device(workspace, q.device, "workspace")
    with torch.cuda.device(q.device):
        rc = fa_fwd_tree(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(),
                         lse.data_ptr(), ctx_len.data_ptr(),
                         None if tree is None else tree.data_ptr(),
                         tree is not None and tree.dim() == 3,
                         None if depths is None else depths.data_ptr(),
                         depths is not None and depths.dim() == 2, softcap,
                         None if slopes is None else slopes.data_ptr(), B, H, Hkv, Tq, Tmax, d,
                         scale, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                         None if status is None else status.data_ptr(), timeout_ns,
                         torch.cuda.current_stream(q.device).cuda_stream)
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_tree")
    return out, lse


def rope_inv_freq(rot_dim: int, base: float = 10000.0, scaling: str | None = None,
                  factor: float = 1.0, original_length: int = 4096, low_turns: float = 1.0,
                  high_turns: float = 32.0, device=None):
    """Radians a position for each of rot_dim/2 pairs, base^(−2i/rot_dim), as the float64 tensor
    that ``rope`` takes.

    Scaled for contexts ``factor`` times longer: ``"linear"`` divides every frequency by it;
    ``"by_parts"`` leaves pairs that make more than ``high_turns`` turns in ``original_length``
    positions, divides those that make fewer than ``low_turns``, and goes from one to the other
    linearly in the number of turns between.
    """
    import torch
    if rot_dim <= 0 or rot_dim % 16 or not base > 0 or not factor > 0:
        raise ValueError("rot_dim must be a positive multiple of 16, base and factor positive")
    f = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":
        if not high_turns > low_turns:
            raise ValueError("high_turns must be above low_turns")
        turns = original_length * f / (2.0 * math.pi)
        keep = ((turns - low_turns) / (high_turns - low_turns)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    elif scaling is not None:
        raise ValueError("scaling must be None, 'linear' or 'by_parts'")
    return f.to("cuda" if device is None else device)


def _check_rows(t, name, B, n, T, d):
    """A bf16 CUDA [B, n, T, d] tensor of any strides that 16-byte vectors can read; its (batch,
    head, token) strides, 0 for a dimension of one."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 4:
        raise ValueError(f"{name} must be a CUDA bfloat16 tensor of four dimensions")
    if tuple(t.shape) != (B, n, T, d):
        raise ValueError(f"{name} must have shape {[B, n, T, d]}")
    s = t.stride()
    strides = tuple(0 if m == 1 else x for m, x in zip((B, n, T), s))
    if (s[3] != 1 and d > 1) or any(x % 8 for x in strides):
        raise ValueError(f"{name} must have a contiguous last dimension and other strides that "
                         "are multiples of 8 elements")
    return strides


def _check_turn(q, inv_freq, positions, B, T, d):
    """The rotary arguments; (rot_dim, whether positions are given for each sequence)."""
    import torch
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dtype != torch.float64 \
            or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous float64 tensor of one dimension")
    _same_device(inv_freq, q.device, "inv_freq")
    rot = 2 * inv_freq.numel()
    if rot % 16 or not 0 < rot <= d:
        raise ValueError(f"inv_freq must hold 8, 16, … {d // 2} frequencies")
    if positions is not None:
        _check_int32(positions, ((T,), (B, T)), q.device, "positions")
    return rot, positions is not None and positions.dim() == 2


def rope(q, k, inv_freq, positions=None, interleaved: bool = False, inverse: bool = False,
         mscale: float = 1.0, out_q=None, out_k=None):
    """Queries [B, H, T, d] and keys [B, Hkv, T, d] (or None) turned by their positions, through
    fa_rope: the first 2·len(inv_freq) dimensions of each head in pairs (i, i + half), or
    (2i, 2i + 1) when ``interleaved``, by position·inv_freq (``rope_inv_freq``), times ``mscale``.

    ``positions``: int32 [T] or [B, T]; None: 0 … T − 1. ``inverse`` turns back: the gradients of q
    and k from those of the results. The inputs may be views of a packed projection; the results
    are contiguous. ``out_q``/``out_k`` may be the (contiguous) inputs themselves. Returns (q, k).
    """
    import torch
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a tensor of shape [B, H, T, d]")
    B, H, T, d = q.shape
    qs = _check_rows(q, "q", B, H, T, d)
    Hkv, ks = 0, (0, 0, 0)
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be a tensor of shape [B, Hkv, T, d]")
        Hkv = k.shape[1]
        ks = _check_rows(k, "k", B, Hkv, T, d)
        _same_device(k, q.device, "k")
    rot, per_batch = _check_turn(q, inv_freq, positions, B, T, d)
    if out_q is None:
        out_q = torch.empty((B, H, T, d), dtype=q.dtype, device=q.device)
    else:
        _check_like(out_q, q, "out_q")
    if k is None:
        if out_k is not None:
            raise ValueError("out_k without k")
    elif out_k is None:
        out_k = torch.empty((B, Hkv, T, d), dtype=q.dtype, device=q.device)
    else:
        _check_like(out_k, k, "out_k")
    with torch.cuda.device(q.device):
        rc = fa_rope(q.data_ptr(), qs, out_q.data_ptr(), None if k is None else k.data_ptr(), ks,
                     None if k is None else out_k.data_ptr(),
                     None if positions is None else positions.data_ptr(), per_batch,
                     inv_freq.data_ptr(), rot, interleaved, inverse, mscale, B, H, Hkv, T, d,
                     torch.cuda.current_stream(q.device).cuda_stream)
    if rc != FA_OK:
        raise FAError(rc, "fa_rope")
    return out_q, out_k


def rope_append(q, k, v, k_cache, v_cache, ctx_len, inv_freq, positions=None,
                interleaved: bool = False, mscale: float = 1.0, out=None):
    """A serving step's new tokens through fa_rope_append: q [B, H, Tq, d] turned and returned, k
    turned and v as it is ([B, Hkv, Tq, d], any strides) written into rows ctx_len[b] … of the
    caches [B, Hkv, Tmax, d].

    ``ctx_len``: int32 [B], the tokens each sequence's cache holds already; negative: an inactive
    sequence, whose result is 0 and whose cache stays. Rows past Tmax are not written.
    ``positions``: int32 [Tq] or [B, Tq]; None: ctx_len[b] + t. The rest as for ``rope``.
    """
    import torch
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a tensor of shape [B, H, Tq, d]")
    B, H, Tq, d = q.shape
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _check(t, n)
        _same_device(t, q.device, n)
    Hkv, Tmax = k_cache.shape[1], k_cache.shape[2]
    if tuple(k_cache.shape) != (B, Hkv, Tmax, d) or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must be [B, Hkv, Tmax, d]")
    qs = _check_rows(q, "q", B, H, Tq, d)
    ks, vs = _check_rows(k, "k", B, Hkv, Tq, d), _check_rows(v, "v", B, Hkv, Tq, d)
    for t, n in ((k, "k"), (v, "v")):
        _same_device(t, q.device, n)
    _check_int32(ctx_len, ((B,),), q.device, "ctx_len")
    rot, per_batch = _check_turn(q, inv_freq, positions, B, Tq, d)
    if out is None:
        out = torch.empty((B, H, Tq, d), dtype=q.dtype, device=q.device)
    else:
        _check_like(out, q, "out")
    with torch.cuda.device(q.device):
        rc = fa_rope_append(q.data_ptr(), qs, out.data_ptr(), k.data_ptr(), ks, v.data_ptr(), vs,
                            k_cache.data_ptr(), v_cache.data_ptr(), ctx_len.data_ptr(),
                            None if positions is None else positions.data_ptr(), per_batch,
                            inv_freq.data_ptr(), rot, interleaved, mscale, B, H, Hkv, Tq, Tmax, d,
                            torch.cuda.current_stream(q.device).cuda_stream)
    if rc != FA_OK:
        raise FAError(rc, "fa_rope_append")
    return out

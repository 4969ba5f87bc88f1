"""Attention with modified scores, new tokens against a cache, and rotary positions: allocation,
argument checks and the calls of libfa.so (include/fa.h).

Short calls are bound by the host, so each check first asks the one expression that holds for good
arguments, and looks for what is wrong only when it does not.
"""

from __future__ import annotations

import functools
import math

import torch

from . import _check
from ._binding import (
    FA_ERR_INVALID_ARG,
    FA_OK,
    FAError,
    fa_bwd_mod_workspace_size,
    fa_bwd_window_workspace_size,
    fa_fwd_tree4_workspace_size,
    fa_fwd_tree_window_workspace_size,
    fa_fwd_tree_workspace_size,
    fa_norm_rope_bwd_workspace_size,
    fa_visible_size,
    fa_visible_window_size,
    lib,
)

_BF16, _FP32, _INT32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
# A device's current stream as an address, and the current device (torch.cuda.current_stream makes
# a Stream object first, 2 µs of a short call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) \
    or (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_functions: dict = {}


def _call(device, name, *args):
    """libfa.so's function ``name`` on args and ``device``'s current stream, with the device current;
    raises on a status. (Truth values go as they are: its argument types take them for ints.)"""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(lib(), name)
    index = device.index
    if index == _current_device():
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc != FA_OK:
        raise FAError(rc, name)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _same_device(t, device, name):
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, as the other tensors")


def _check_on(t, device, name):
    """A contiguous bf16 CUDA tensor of four dimensions on ``device``."""
    if type(t) is torch.Tensor and t.dtype is _BF16 and t.is_cuda and t.device == device \
            and t.dim() == 4 and t.is_contiguous():
        return
    _check(t, name)
    _same_device(t, device, name)


def _check_like(t, ref, name):
    _check_on(t, ref.device, name)
    if t.shape != ref.shape:
        raise ValueError(f"{name} must have shape {list(ref.shape)}")


def _check_int32(t, shapes, device, name):
    if not isinstance(t, torch.Tensor) or t.dtype is not _INT32 or t.shape not in shapes \
            or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name} must be a contiguous CUDA int32 tensor of shape "
                         + " or ".join(str(list(s)) for s in shapes))
    if t.device != device:
        _same_device(t, device, name)


def _check_fp32(t, shape, device, name):
    if not isinstance(t, torch.Tensor) or t.dtype is not _FP32 or t.shape != shape \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {list(shape)}")
    _same_device(t, device, name)


def _check_workspace(t, device):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    _same_device(t, device, "workspace")


def _check_status(t, device):
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or t.dtype is not _INT32 or t.numel() < 1 or not t.is_cuda:
        raise ValueError("status must be a CUDA int32 tensor of one element")
    _same_device(t, device, "status")


# --------------------------------------------------------------------------- who sees whom

class Visible:
    """Who sees whom in a batch, made by ``visible``: an opaque device buffer that ``fwd_mod`` and
    ``bwd_mod`` calls of the same B and T read."""

    __slots__ = ("buffer", "B", "T", "causal", "window", "sinks")

    def __init__(self, buffer, B: int, T: int, causal: bool, window: int = 0, sinks: int = 0):
        self.buffer, self.B, self.T, self.causal = buffer, B, T, causal
        self.window, self.sinks = window, sinks


def _check_window(window, sinks, most):
    """A sliding window (0: none) and its sinks."""
    if type(window) is not int or type(sinks) is not int or window < 0 or sinks < 0:
        raise ValueError("window and sinks must be whole numbers of at least 0")
    if sinks and not window:
        raise ValueError("sinks without a window: without one every token stays visible")
    if window > 0x7FFFFFFF or sinks > most:
        raise ValueError(f"window must be below 2**31, sinks at most {most}")


@functools.lru_cache(maxsize=256)
def _visible_bytes(B, T, window, sinks):
    """fa_visible_size or fa_visible_window_size, functions of their arguments alone."""
    n = fa_visible_window_size(B, T, window, sinks) if window else fa_visible_size(B, T)
    if n == 0:
        raise FAError(FA_ERR_INVALID_ARG, "fa_visible_size")
    return n


def visible(B: int, T: int, causal: bool = True, doc_ids=None, prefix_len=None, device=None,
            buffer=None, window: int = 0, sinks: int = 0) -> Visible:
    """The visibility of a batch of B sequences of T tokens, for every layer's ``fwd_mod`` and
    ``bwd_mod``.

    ``doc_ids`` (int32 [B, T]): a document is a maximal run of equal ids and sees itself only; a
    negative id is padding, which sees nothing and is seen by nothing. ``causal``: key j is
    visible to query i when j ≤ i or j is one of the first ``prefix_len`` tokens of their document
    (int32 [B], or [B, T] with each token holding its document's). ``window`` > 0 (causal, no
    prefixes): a token sees the last ``window`` tokens of its document, itself among them, and the
    document's first ``sinks`` (at most 1024). ``buffer``, a uint8 CUDA tensor of fa_visible_size(B, T)
    bytes (with a window fa_visible_window_size(B, T, window, sinks)), may be given to reuse it.
    """
    _check_window(window, sinks, 1024)
    if window and (not causal or prefix_len is not None):
        raise ValueError("a window is causal and takes no prefixes")
    if device is None:
        device = next((t.device for t in (doc_ids, prefix_len, buffer) if t is not None), "cuda")
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("the visibility lives on a CUDA device")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    if doc_ids is not None:
        _check_int32(doc_ids, ((B, T),), device, "doc_ids")
    if prefix_len is not None:
        _check_int32(prefix_len, ((B,), (B, T)), device, "prefix_len")
    need = _visible_bytes(B, T, window, sinks)
    if buffer is None:
        buffer = torch.empty(need, dtype=_U8, device=device)
    elif not isinstance(buffer, torch.Tensor) or buffer.dtype is not _U8 or not buffer.is_contiguous():
        raise ValueError("buffer must be a contiguous uint8 CUDA tensor")
    _same_device(buffer, device, "buffer")
    if window:
        _call(device, "fa_visible_window", _ptr(doc_ids), window, sinks, buffer.data_ptr(),
              buffer.numel(), B, T)
        return Visible(buffer, B, T, True, window, sinks)
    _call(device, "fa_visible", _ptr(doc_ids), _ptr(prefix_len),
          prefix_len is not None and prefix_len.dim() == 2, causal, buffer.data_ptr(),
          buffer.numel(), B, T)
    return Visible(buffer, B, T, bool(causal))


# ---------------------------------------------------------------- attention, modified scores

def _check_mod(q, k, v, seen, causal, slopes):
    """Shapes, devices and masks of a modified-score call; q's shape, the key heads, and the causal
    flag that holds."""
    _check(q, "q")
    device = q.device
    _check_on(k, device, "k")
    _check_on(v, device, "v")
    B, H, T, d = q.shape
    Bk, Hkv, Tk, dk = shape = k.shape
    if v.shape != shape or Bk != B or Tk != T or dk != d or Hkv == 0 or H % Hkv:
        raise ValueError("q must be [B, H, T, d] and k, v [B, Hkv, T, d] with Hkv a divisor of H")
    if slopes is not None:
        _check_fp32(slopes, (H,), device, "slopes")
    if seen is None:
        return B, H, T, d, Hkv, True if causal is None else causal
    if not isinstance(seen, Visible):
        raise TypeError("visible must be what visible() returned")
    if seen.B != B or seen.T != T:
        raise ValueError(f"visible is for B {seen.B}, T {seen.T}, the tensors for B {B}, T {T}")
    if causal is not None and bool(causal) != seen.causal:
        raise ValueError("causal differs from what visible was made with")
    _same_device(seen.buffer, device, "visible")
    return B, H, T, d, Hkv, seen.causal


def fwd_mod(q, k, v, visible=None, causal: bool | None = None, softcap: float = 0.0, slopes=None,
            scale: float | None = None, out=None, lse=None, rest=None, status=None,
            timeout_ns: int = 0):
    """Attention with modified scores through fa_fwd_mod: z = scale·q·k, capped to
    softcap·tanh(z / softcap) when ``softcap`` > 0, lowered by slopes[h]·|i − j| when ``slopes``
    (float32 [H]) is given; softmax over the visible keys.

    q is [B, H, T, d], k and v [B, Hkv, T, d] with Hkv a divisor of H. ``visible`` (from
    ``visible()``) says who sees whom; without it ``causal`` does (None: causal). Returns
    (o, lse); a row that sees no key has o = 0 and lse = −inf. ``rest``, a tensor like q, is
    written with what o's rounding to bf16 leaves out, for ``bwd_mod``.
    """
    B, H, T, d, Hkv, causal = _check_mod(q, k, v, visible, causal, slopes)
    device = q.device
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_like(out, q, "out")
    if lse is None:
        lse = torch.empty((B, H, T), dtype=_FP32, device=device)
    else:
        _check_fp32(lse, (B, H, T), device, "lse")
    if rest is not None:
        _check_like(rest, q, "rest")
    _check_status(status, device)
    if visible is not None and visible.window:
        _call(device, "fa_fwd_window", q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
              lse.data_ptr(), _ptr(rest), visible.buffer.data_ptr(), visible.window, visible.sinks,
              softcap, _ptr(slopes), B, H, Hkv, T, d, scale, _ptr(status), timeout_ns)
        return out, lse
    _call(device, "fa_fwd_mod", q.data_ptr(), k.data_ptr(), v.data_ptr(),
          out.data_ptr(), lse.data_ptr(), _ptr(rest), None if visible is None else visible.buffer.data_ptr(),
          causal, softcap, _ptr(slopes), B, H, Hkv, T, d, scale, _ptr(status), timeout_ns)
    return out, lse


def bwd_mod_workspace(B: int, H: int, Hkv: int, T: int, d: int, device=None, window: int = 0,
                      sinks: int = 0):
    """A uint8 CUDA tensor large enough to serve as ``bwd_mod``'s workspace (with a visibility that has
    this window and these sinks)."""
    return torch.empty(_bwd_bytes(B, H, Hkv, T, d, window, sinks), dtype=_U8,
                       device="cuda" if device is None else device)


@functools.lru_cache(maxsize=256)
def _bwd_bytes(B, H, Hkv, T, d, window, sinks):
    """fa_bwd_mod_workspace_size or fa_bwd_window_workspace_size, functions of their arguments alone."""
    n = (fa_bwd_window_workspace_size(B, H, Hkv, T, d, window, sinks) if window
         else fa_bwd_mod_workspace_size(B, H, Hkv, T, d))
    if n == 0:
        raise FAError(FA_ERR_INVALID_ARG, "fa_bwd_mod_workspace_size")
    return n


def bwd_mod(q, k, v, o, lse, do, visible=None, causal: bool | None = None, softcap: float = 0.0,
            slopes=None, scale: float | None = None, rest=None, dq=None, dk=None, dv=None,
            workspace=None, status=None, timeout_ns: int = 0):
    """Gradients of ``fwd_mod`` through fa_bwd_mod: (dq [B, H, T, d], dk, dv [B, Hkv, T, d]), from
    its outputs ``o`` and ``lse`` and the gradient ``do`` of o; the other arguments as there. With
    the ``rest`` that the forward wrote, dq and dk do not suffer from o's rounding (it shows where
    one key takes most of a row's weight).
    ``workspace`` (see ``bwd_mod_workspace``) may be passed to reuse it."""
    B, H, T, d, Hkv, causal = _check_mod(q, k, v, visible, causal, slopes)
    device = q.device
    _check_like(o, q, "o")
    _check_like(do, q, "do")
    _check_fp32(lse, (B, H, T), device, "lse")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if dq is None:
        dq = torch.empty_like(q)
    else:
        _check_like(dq, q, "dq")
    if dk is None:
        dk = torch.empty_like(k)
    else:
        _check_like(dk, k, "dk")
    if dv is None:
        dv = torch.empty_like(v)
    else:
        _check_like(dv, v, "dv")
    if workspace is None:
        workspace = bwd_mod_workspace(B, H, Hkv, T, d, device, *(() if visible is None else
                                                                 (visible.window, visible.sinks)))
    else:
        _check_workspace(workspace, device)
    if rest is not None:
        _check_like(rest, q, "rest")
    _check_status(status, device)
    if visible is not None and visible.window:
        _call(device, "fa_bwd_window", q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
              do.data_ptr(), lse.data_ptr(), _ptr(rest), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
              workspace.data_ptr(), workspace.numel() * workspace.element_size(),
              visible.buffer.data_ptr(), visible.window, visible.sinks, softcap, _ptr(slopes),
              B, H, Hkv, T, d, scale, _ptr(status), timeout_ns)
        return dq, dk, dv
    _call(device, "fa_bwd_mod", q.data_ptr(), k.data_ptr(), v.data_ptr(),
          o.data_ptr(), do.data_ptr(), lse.data_ptr(), _ptr(rest), dq.data_ptr(), dk.data_ptr(),
          dv.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
          None if visible is None else visible.buffer.data_ptr(), causal, softcap, _ptr(slopes),
          B, H, Hkv, T, d, scale, _ptr(status), timeout_ns)
    return dq, dk, dv


# -------------------------------------------------------------- new tokens against a cache

def fwd_tree_workspace(B: int, H: int, Hkv: int, Tq: int, Tmax: int, d: int, device=None,
                       window: int = 0, sinks: int = 0):
    """A uint8 CUDA tensor large enough to serve as ``fwd_tree``'s workspace."""
    _check_window(window, sinks, 0x7FFFFFFF)
    device = torch.device("cuda" if device is None else device)
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return torch.empty(_tree_bytes(B, H, Hkv, Tq, Tmax, d, window, sinks, device.index), dtype=_U8,
                       device=device)


@functools.lru_cache(maxsize=256)
def _tree_bytes(B, H, Hkv, Tq, Tmax, d, window, sinks, index):
    """fa_fwd_tree_workspace_size on device ``index``, a function of its arguments alone."""
    with torch.cuda.device(index):
        n = (fa_fwd_tree_window_workspace_size(B, H, Hkv, Tq, Tmax, d, window, sinks) if window
             else fa_fwd_tree_workspace_size(B, H, Hkv, Tq, Tmax, d))
    if n == 0:
        raise FAError(FA_ERR_INVALID_ARG, "fa_fwd_tree_workspace_size")
    return n


def _check_tree(ctx_len, tree, depths, slopes, B, H, Tq, device):
    """The context lengths of a batch, and what its new tokens see of one another."""
    _check_int32(ctx_len, ((B,),), device, "ctx_len")
    if tree is not None:
        if not isinstance(tree, torch.Tensor) or tree.dtype not in (_U8, torch.bool) \
                or not tree.is_contiguous() or tree.shape not in ((Tq, Tq), (B, Tq, Tq)):
            raise ValueError(f"tree must be a contiguous uint8 or bool tensor of shape "
                             f"[{Tq}, {Tq}] or [{B}, {Tq}, {Tq}]")
        _same_device(tree, device, "tree")
    if depths is not None:
        _check_int32(depths, ((Tq,), (B, Tq)), device, "depths")
    if slopes is not None:
        _check_fp32(slopes, (H,), device, "slopes")


def fwd_tree(q, k_cache, v_cache, ctx_len, tree=None, depths=None, softcap: float = 0.0,
             slopes=None, scale: float | None = None, out=None, lse=None, workspace=None,
             status=None, timeout_ns: int = 0, window: int = 0, sinks: int = 0):
    """New tokens q [B, H, Tq, d] against caches [B, Hkv, Tmax, d] through fa_fwd_tree: sequence b
    holds ``ctx_len[b]`` tokens (int32 [B]; negative: inactive) and behind them, already written
    (``rope_append``), its Tq new ones.

    A new token sees the whole context and, of the new tokens, those where ``tree`` (uint8 or bool
    [Tq, Tq] or [B, Tq, Tq], nonzero = row t sees token s) says so; without it a chain: itself and
    the ones before. ``softcap`` and ``slopes`` as for ``fwd_mod``, the bias measured between
    positions ctx_len[b] + ``depths`` (int32 [Tq] or [B, Tq]; None: 0, 1, …). With ``window`` > 0 a
    token sees, of these, the rows less than ``window`` positions behind its own and those at positions
    below ``sinks``; the other rows of the cache are not read. Returns (o, lse); a token that sees
    nothing has o = 0 and lse = −inf. ``workspace``: see ``fwd_tree_workspace``.
    """
    if window or sinks:
        _check_window(window, sinks, 0x7FFFFFFF)
    _check(q, "q")
    device = q.device
    _check_on(k_cache, device, "k_cache")
    _check_on(v_cache, device, "v_cache")
    B, H, Tq, d = q.shape
    Bk, Hkv, Tmax, dk = shape = k_cache.shape
    if v_cache.shape != shape or Bk != B or dk != d or Hkv == 0 or H % Hkv:
        raise ValueError("q must be [B, H, Tq, d] and the caches [B, Hkv, Tmax, d] with Hkv a "
                         "divisor of H")
    _check_tree(ctx_len, tree, depths, slopes, B, H, Tq, device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_like(out, q, "out")
    if lse is None:
        lse = torch.empty((B, H, Tq), dtype=_FP32, device=device)
    else:
        _check_fp32(lse, (B, H, Tq), device, "lse")
    if workspace is None:
        need = _tree_bytes(B, H, Hkv, Tq, Tmax, d, window, sinks, device.index)
        if need > 1:
            workspace = torch.empty(need, dtype=_U8, device=device)
    else:
        _check_workspace(workspace, device)
        need = workspace.numel() * workspace.element_size()
    _check_status(status, device)
    if window:
        _call(device, "fa_fwd_tree_window", q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
              out.data_ptr(), lse.data_ptr(), ctx_len.data_ptr(), _ptr(tree),
              tree is not None and tree.dim() == 3, _ptr(depths),
              depths is not None and depths.dim() == 2, window, sinks, softcap, _ptr(slopes), B, H, Hkv,
              Tq, Tmax, d, scale, _ptr(workspace), need, _ptr(status), timeout_ns)
        return out, lse
    _call(device, "fa_fwd_tree", q.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), out.data_ptr(), lse.data_ptr(), ctx_len.data_ptr(), _ptr(tree),
          tree is not None and tree.dim() == 3, _ptr(depths),
          depths is not None and depths.dim() == 2, softcap, _ptr(slopes), B, H, Hkv, Tq, Tmax, d,
          scale, _ptr(workspace), need, _ptr(status), timeout_ns)
    return out, lse


# ------------------------------------------------------------------------ rotary positions

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


def _check_rows(t, name, shape, device):
    """A bf16 CUDA tensor of ``shape`` [B, n, T, d] and any strides that 16-byte vectors can read;
    its (batch, head, token) strides, 0 for a dimension of one."""
    if not (type(t) is torch.Tensor and t.dtype is _BF16 and t.shape == shape
            and t.device == device and t.is_cuda):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda or t.dtype is not _BF16 or t.dim() != 4:
            raise ValueError(f"{name} must be a CUDA bfloat16 tensor of four dimensions")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {list(shape)}")
        _same_device(t, device, name)
    sb, sh, st, sd = t.stride()
    if shape[0] == 1:
        sb = 0
    if shape[1] == 1:
        sh = 0
    if shape[2] == 1:
        st = 0
    if sd != 1 or (sb | sh | st) & 7:
        raise ValueError(f"{name} must have a contiguous last dimension and other strides that "
                         "are multiples of 8 elements")
    return sb, sh, st


def _check_turn(inv_freq, positions, B, T, d, device):
    """The rotary arguments; (rot_dim, whether positions are given for each sequence)."""
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dtype is not torch.float64 \
            or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous float64 tensor of one dimension")
    _same_device(inv_freq, device, "inv_freq")
    rot = 2 * inv_freq.numel()
    if rot % 16 or not 0 < rot <= d:
        raise ValueError(f"inv_freq must hold 8, 16, … {d // 2} frequencies")
    if positions is None:
        return rot, False
    _check_int32(positions, ((T,), (B, T)), device, "positions")
    return rot, positions.dim() == 2


def rope(q, k, inv_freq, positions=None, interleaved: bool = False, inverse: bool = False,
         mscale: float = 1.0, out_q=None, out_k=None):
    """Queries [B, H, T, d] and keys [B, Hkv, T, d] (or None) turned by their positions, through
    fa_rope: the first 2·len(inv_freq) dimensions of each head in pairs (i, i + half), or
    (2i, 2i + 1) when ``interleaved``, by position·inv_freq (``rope_inv_freq``), times ``mscale``.

    ``positions``: int32 [T] or [B, T]; None: 0 … T − 1. ``inverse`` turns back: the gradients of q
    and k from those of the results. The inputs may be views of a packed projection; the results
    are contiguous. ``out_q``/``out_k`` may be the (contiguous) inputs themselves. Returns (q, k).
    """
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a tensor of shape [B, H, T, d]")
    shape, device = q.shape, q.device
    B, H, T, d = shape
    qs = _check_rows(q, "q", shape, device)
    if k is None:
        Hkv, ks = 0, (0, 0, 0)
        if out_k is not None:
            raise ValueError("out_k without k")
    else:
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be a tensor of shape [B, Hkv, T, d]")
        Hkv = k.shape[1]
        ks = _check_rows(k, "k", (B, Hkv, T, d), device)
        if out_k is None:
            out_k = torch.empty((B, Hkv, T, d), dtype=_BF16, device=device)
        else:
            _check_like(out_k, k, "out_k")
    rot, per_batch = _check_turn(inv_freq, positions, B, T, d, device)
    if out_q is None:
        out_q = torch.empty(shape, dtype=_BF16, device=device)
    else:
        _check_like(out_q, q, "out_q")
    _call(device, "fa_rope", q.data_ptr(), *qs, out_q.data_ptr(), _ptr(k), *ks,
          _ptr(out_k), _ptr(positions), per_batch, inv_freq.data_ptr(), rot, interleaved, inverse,
          mscale, B, H, Hkv, T, d)
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
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a tensor of shape [B, H, Tq, d]")
    shape, device = q.shape, q.device
    B, H, Tq, d = shape
    _check_on(k_cache, device, "k_cache")
    _check_on(v_cache, device, "v_cache")
    Bk, Hkv, Tmax, dk = cache = k_cache.shape
    if v_cache.shape != cache or Bk != B or dk != d:
        raise ValueError("k_cache and v_cache must be [B, Hkv, Tmax, d]")
    qs = _check_rows(q, "q", shape, device)
    new = (B, Hkv, Tq, d)
    ks, vs = _check_rows(k, "k", new, device), _check_rows(v, "v", new, device)
    _check_int32(ctx_len, ((B,),), device, "ctx_len")
    rot, per_batch = _check_turn(inv_freq, positions, B, Tq, d, device)
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=device)
    else:
        _check_like(out, q, "out")
    _call(device, "fa_rope_append", q.data_ptr(), *qs, out.data_ptr(),
          k.data_ptr(), *ks, v.data_ptr(), *vs, k_cache.data_ptr(), v_cache.data_ptr(),
          ctx_len.data_ptr(), _ptr(positions), per_batch, inv_freq.data_ptr(), rot, interleaved,
          mscale, B, H, Hkv, Tq, Tmax, d)
    return out


# -------------------------------------------------------- head norms with rotary positions

def _check_weight(t, d, device, name):
    if not (isinstance(t, torch.Tensor) and t.dtype is _FP32 and t.shape == (d,) and t.device == device
            and t.is_contiguous()):
        _check_fp32(t, (d,), device, name)


def _check_four(t, name, heads):
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        raise ValueError(f"{name} must be a tensor of shape [B, {heads}, T, d]")


def norm_rope(q, k, q_weight, k_weight, inv_freq, positions=None, interleaved: bool = False,
              mscale: float = 1.0, eps: float = 1e-6, out_q=None, out_k=None):
    """Queries [B, H, T, d] and keys [B, Hkv, T, d] (or None, with ``k_weight`` None) normed and turned
    in one pass, through fa_norm_rope: each head's row is divided by √(mean of its squares + eps),
    multiplied by its weight (float32 [d], one for queries and one for keys) and turned as ``rope``
    does. Inputs may be views of a packed projection; ``out_q``/``out_k`` may be the (contiguous)
    inputs themselves. Returns (q, k)."""
    _check_four(q, "q", "H")
    shape, device = q.shape, q.device
    B, H, T, d = shape
    qs = _check_rows(q, "q", shape, device)
    _check_weight(q_weight, d, device, "q_weight")
    if k is None:
        Hkv, ks = 0, (0, 0, 0)
        if out_k is not None or k_weight is not None:
            raise ValueError("out_k or k_weight without k")
    else:
        _check_four(k, "k", "Hkv")
        Hkv = k.shape[1]
        ks = _check_rows(k, "k", (B, Hkv, T, d), device)
        _check_weight(k_weight, d, device, "k_weight")
        if out_k is None:
            out_k = torch.empty((B, Hkv, T, d), dtype=_BF16, device=device)
        else:
            _check_like(out_k, k, "out_k")
    rot, per_batch = _check_turn(inv_freq, positions, B, T, d, device)
    if out_q is None:
        out_q = torch.empty(shape, dtype=_BF16, device=device)
    else:
        _check_like(out_q, q, "out_q")
    _call(device, "fa_norm_rope", q.data_ptr(), *qs, out_q.data_ptr(), _ptr(k), *ks, _ptr(out_k),
          q_weight.data_ptr(), _ptr(k_weight), eps, _ptr(positions), per_batch, inv_freq.data_ptr(),
          rot, interleaved, mscale, B, H, Hkv, T, d)
    return out_q, out_k


def norm_rope_bwd_workspace(d: int, device=None):
    """A uint8 CUDA tensor that serves as ``norm_rope_bwd``'s workspace for head dim d, at any size."""
    n = fa_norm_rope_bwd_workspace_size(d)
    if n == 0:
        raise FAError(FA_ERR_INVALID_ARG, "fa_norm_rope_bwd_workspace_size")
    return torch.empty(n, dtype=_U8, device="cuda" if device is None else device)


def norm_rope_bwd(gq, gk, q, k, q_weight, k_weight, inv_freq, positions=None, interleaved: bool = False,
                  mscale: float = 1.0, eps: float = 1e-6, dq=None, dk=None, dq_weight=None,
                  dk_weight=None, workspace=None):
    """Gradients of ``norm_rope`` through fa_norm_rope_bwd, from those of its results, ``gq`` and
    ``gk`` (as ``bwd_mod`` returns them; any strides), and its inputs; the other arguments as there.
    Returns (dq, dk, dq_weight, dk_weight): contiguous rows in bf16 and float32 [d] sums over all rows
    (added in a fixed order: the same bits every time; every row counts, so those of padding must hold
    numbers). gk, k and k_weight may be None together.
    ``dq``/``dk`` may be the (contiguous) ``gq``/``gk``; ``workspace``: see ``norm_rope_bwd_workspace``.
    """
    _check_four(q, "q", "H")
    shape, device = q.shape, q.device
    B, H, T, d = shape
    qs = _check_rows(q, "q", shape, device)
    gqs = _check_rows(gq, "gq", shape, device)
    _check_weight(q_weight, d, device, "q_weight")
    if k is None:
        Hkv, ks, gks = 0, (0, 0, 0), (0, 0, 0)
        if any(x is not None for x in (gk, k_weight, dk, dk_weight)):
            raise ValueError("gk, k_weight, dk or dk_weight without k")
    else:
        _check_four(k, "k", "Hkv")
        Hkv = k.shape[1]
        kshape = (B, Hkv, T, d)
        ks = _check_rows(k, "k", kshape, device)
        gks = _check_rows(gk, "gk", kshape, device)
        _check_weight(k_weight, d, device, "k_weight")
        if dk is None:
            dk = torch.empty(kshape, dtype=_BF16, device=device)
        else:
            _check_like(dk, k, "dk")
        if dk_weight is None:
            dk_weight = torch.empty(d, dtype=_FP32, device=device)
        else:
            _check_weight(dk_weight, d, device, "dk_weight")
    rot, per_batch = _check_turn(inv_freq, positions, B, T, d, device)
    if dq is None:
        dq = torch.empty(shape, dtype=_BF16, device=device)
    else:
        _check_like(dq, q, "dq")
    if dq_weight is None:
        dq_weight = torch.empty(d, dtype=_FP32, device=device)
    else:
        _check_weight(dq_weight, d, device, "dq_weight")
    if workspace is None:
        workspace = norm_rope_bwd_workspace(d, device=device)
    else:
        _check_workspace(workspace, device)
    _call(device, "fa_norm_rope_bwd", gq.data_ptr(), *gqs, q.data_ptr(), *qs, dq.data_ptr(), _ptr(gk),
          *gks, _ptr(k), *ks, _ptr(dk), q_weight.data_ptr(), _ptr(k_weight), dq_weight.data_ptr(),
          _ptr(dk_weight), eps, _ptr(positions), per_batch, inv_freq.data_ptr(), rot, interleaved,
          mscale, B, H, Hkv, T, d, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return dq, dk, dq_weight, dk_weight


def norm_rope_append(q, k, v, q_weight, k_weight, k_cache, v_cache, ctx_len, inv_freq, positions=None,
                     interleaved: bool = False, mscale: float = 1.0, eps: float = 1e-6, out=None):
    """A serving step's new tokens through fa_norm_rope_append: ``rope_append`` with the norm of
    ``norm_rope`` in front of the rotation (v goes into its cache as it is)."""
    _check_four(q, "q", "H")
    shape, device = q.shape, q.device
    B, H, Tq, d = shape
    _check_on(k_cache, device, "k_cache")
    _check_on(v_cache, device, "v_cache")
    Bk, Hkv, Tmax, dk = cache = k_cache.shape
    if v_cache.shape != cache or Bk != B or dk != d:
        raise ValueError("k_cache and v_cache must be [B, Hkv, Tmax, d]")
    qs = _check_rows(q, "q", shape, device)
    new = (B, Hkv, Tq, d)
    ks, vs = _check_rows(k, "k", new, device), _check_rows(v, "v", new, device)
    _check_weight(q_weight, d, device, "q_weight")
    _check_weight(k_weight, d, device, "k_weight")
    _check_int32(ctx_len, ((B,),), device, "ctx_len")
    rot, per_batch = _check_turn(inv_freq, positions, B, Tq, d, device)
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=device)
    else:
        _check_like(out, q, "out")
    _call(device, "fa_norm_rope_append", q.data_ptr(), *qs, out.data_ptr(), k.data_ptr(), *ks,
          v.data_ptr(), *vs, q_weight.data_ptr(), k_weight.data_ptr(), eps, k_cache.data_ptr(),
          v_cache.data_ptr(), ctx_len.data_ptr(), _ptr(positions), per_batch, inv_freq.data_ptr(), rot,
          interleaved, mscale, B, H, Hkv, Tq, Tmax, d)
    return out


# ------------------------------------------------------------------- a cache held in 4 bits

class Cache4:
    """Keys and values of B sequences in 4 bits: codes, uint8 [B, Hkv, Tmax, d/2], and scales, bfloat16
    [B, Hkv, Tmax, d/32], of each (the format: include/fa.h). ``cache4`` makes an empty one."""

    __slots__ = ("k_codes", "k_scales", "v_codes", "v_scales", "shape", "device")

    def __init__(self, k_codes, k_scales, v_codes, v_scales):
        if not isinstance(k_codes, torch.Tensor) or k_codes.dim() != 4 or not k_codes.is_cuda:
            raise ValueError("k_codes must be a CUDA tensor of shape [B, Hkv, Tmax, d/2]")
        B, Hkv, Tmax, half = codes = k_codes.shape
        if half not in (32, 64) or Tmax % 8:
            raise ValueError("d must be 64 or 128 and Tmax a multiple of 8")
        scales, device = (B, Hkv, Tmax, half // 16), k_codes.device
        for t, shape, dtype, name in ((k_codes, codes, _U8, "k_codes"), (k_scales, scales, _BF16, "k_scales"),
                                      (v_codes, codes, _U8, "v_codes"), (v_scales, scales, _BF16, "v_scales")):
            if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape \
                    or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)}")
            if t.device != device:
                _same_device(t, device, name)
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.shape, self.device = (B, Hkv, Tmax, 2 * half), device

    def _ptrs(self):
        return (self.k_codes.data_ptr(), self.k_scales.data_ptr(), self.v_codes.data_ptr(),
                self.v_scales.data_ptr())


def cache4(B: int, Hkv: int, Tmax: int, d: int, device=None) -> Cache4:
    """An empty 4-bit cache for B sequences of up to Tmax tokens (a multiple of 8): every row zeros."""
    device = torch.device("cuda" if device is None else device)
    if d not in (64, 128) or Tmax % 8:
        raise ValueError("d must be 64 or 128 and Tmax a multiple of 8")
    codes = [torch.full((B, Hkv, Tmax, d // 2), 0x88, dtype=_U8, device=device) for _ in range(2)]
    scales = [torch.zeros((B, Hkv, Tmax, d // 32), dtype=_BF16, device=device) for _ in range(2)]
    return Cache4(codes[0], scales[0], codes[1], scales[1])


def _check_cache4(cache):
    if not isinstance(cache, Cache4):
        raise TypeError("cache must be a Cache4")
    return cache.shape


def append4(k, v, cache, ctx_len):
    """A serving step's new keys (turned already) and values [B, Hkv, Tq, d] (any strides) into rows
    ctx_len[b] … of a 4-bit cache, through fa_append4. ``ctx_len``: int32 [B]; negative: an inactive
    sequence, whose rows stay. Rows past Tmax are not written."""
    B, Hkv, Tmax, d = _check_cache4(cache)
    _check_four(k, "k", "Hkv")
    device, Tq = cache.device, k.shape[2]
    new = (B, Hkv, Tq, d)
    ks, vs = _check_rows(k, "k", new, device), _check_rows(v, "v", new, device)
    _check_int32(ctx_len, ((B,),), device, "ctx_len")
    _call(device, "fa_append4", k.data_ptr(), *ks, v.data_ptr(), *vs, *cache._ptrs(),
          ctx_len.data_ptr(), B, Hkv, Tq, Tmax, d)


def read4(cache, start, n: int, out_k=None, out_v=None):
    """Rows start[b] … start[b] + n − 1 (int32 [B]) of a 4-bit cache as the bf16 values they stand for,
    through fa_read4: (k, v), [B, Hkv, n, d]. Rows past Tmax, and all of a negative start, are zeros."""
    B, Hkv, Tmax, d = _check_cache4(cache)
    device, shape = cache.device, (B, Hkv, n, d)
    _check_int32(start, ((B,),), device, "start")
    outs = []
    for t, name in ((out_k, "out_k"), (out_v, "out_v")):
        if t is None:
            t = torch.empty(shape, dtype=_BF16, device=device)
        else:
            _check_on(t, device, name)
            if t.shape != shape:
                raise ValueError(f"{name} must have shape {list(shape)}")
        outs.append(t)
    _call(device, "fa_read4", *cache._ptrs(), start.data_ptr(), outs[0].data_ptr(), outs[1].data_ptr(),
          B, Hkv, n, Tmax, d)
    return outs[0], outs[1]


@functools.lru_cache(maxsize=256)
def _tree4_bytes(B, H, Hkv, Tq, Tmax, d, window, sinks, index):
    """fa_fwd_tree4_workspace_size on device ``index``, a function of its arguments alone."""
    with torch.cuda.device(index):
        n = fa_fwd_tree4_workspace_size(B, H, Hkv, Tq, Tmax, d, window, sinks)
    if n == 0:
        raise FAError(FA_ERR_INVALID_ARG, "fa_fwd_tree4_workspace_size")
    return n


def fwd_tree4_workspace(B: int, H: int, Hkv: int, Tq: int, Tmax: int, d: int, device=None,
                        window: int = 0, sinks: int = 0):
    """A uint8 CUDA tensor large enough to serve as ``fwd_tree4``'s workspace."""
    _check_window(window, sinks, 0x7FFFFFFF)
    device = torch.device("cuda" if device is None else device)
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return torch.empty(_tree4_bytes(B, H, Hkv, Tq, Tmax, d, window, sinks, device.index), dtype=_U8,
                       device=device)


def fwd_tree4(q, cache, ctx_len, tree=None, depths=None, softcap: float = 0.0, slopes=None,
              scale: float | None = None, out=None, lse=None, workspace=None, status=None,
              timeout_ns: int = 0, window: int = 0, sinks: int = 0):
    """``fwd_tree`` over a 4-bit cache, through fa_fwd_tree4: new tokens q [B, H, Tq, d] against the
    ctx_len[b] tokens of their sequence and one another, whose keys and values ``append4`` has written
    behind them. Every other argument, the window included, and the results as there; keys and values are
    what the codes stand for (``read4``), exactly. (More than 16 rows, H / Hkv · Tq, go in blocks of 16
    that each read the cache.)"""
    _check(q, "q")
    device = q.device
    Bk, Hkv, Tmax, dk = _check_cache4(cache)
    if window or sinks:
        _check_window(window, sinks, 0x7FFFFFFF)
    B, H, Tq, d = q.shape
    if Bk != B or dk != d or Hkv == 0 or H % Hkv:
        raise ValueError("q must be [B, H, Tq, d] and the cache for [B, Hkv, Tmax, d] with Hkv a divisor "
                         "of H")
    if cache.device != device:
        raise ValueError(f"cache must be on {device}, as the other tensors")
    _check_tree(ctx_len, tree, depths, slopes, B, H, Tq, device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_like(out, q, "out")
    if lse is None:
        lse = torch.empty((B, H, Tq), dtype=_FP32, device=device)
    else:
        _check_fp32(lse, (B, H, Tq), device, "lse")
    if workspace is None:
        need = _tree4_bytes(B, H, Hkv, Tq, Tmax, d, window, sinks, device.index)
        if need > 1:
            workspace = torch.empty(need, dtype=_U8, device=device)
    else:
        _check_workspace(workspace, device)
        need = workspace.numel() * workspace.element_size()
    _check_status(status, device)
    _call(device, "fa_fwd_tree4", q.data_ptr(), *cache._ptrs(), out.data_ptr(), lse.data_ptr(),
          ctx_len.data_ptr(), _ptr(tree), tree is not None and tree.dim() == 3, _ptr(depths),
          depths is not None and depths.dim() == 2, window, sinks, softcap, _ptr(slopes), B, H, Hkv, Tq,
          Tmax, d, scale, _ptr(workspace), need, _ptr(status), timeout_ns)
    return out, lse

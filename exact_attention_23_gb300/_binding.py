"""ctypes binding of libfa.so (include/fa.h), with the same names as the C ABI.

Argument marshalling only: every step of the attention computation runs in the CUDA
kernels of libfa.so. PyTorch is used to own device memory and to name the stream.
There is no fallback: if the library is missing, every call raises.
"""

from __future__ import annotations

import ctypes
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libfa.so")

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_MISALIGNED = 2
FA_ERR_UNSUPPORTED_DEVICE = 3
FA_ERR_LAUNCH = 4
FA_ERR_TIMEOUT = 5
FA_FLAG_TEST_STARVE_Q = 1
FA_FLAG_TEST_STARVE_LATER_Q = 2
FA_FLAG_CTA_PAIR = 4
FA_BWD_NOALLOC_SCRATCH_BYTES = 33554432

# Every symbol include/fa.h declares.
EXPORTS = ("fa_fwd", "fa_fwd_ex", "fa_fwd_fp8", "fa_fwd_host_workspace_size", "fa_fwd_host", "fa_fwd_kv_workspace_size", "fa_fwd_kv",
           "fa_fwd_block_sparse", "fa_bwd_workspace_size", "fa_bwd", "fa_bwd_ex",
           "fa_bwd_noalloc", "fa_visible_size", "fa_visible", "fa_fwd_mod", "fa_bwd_mod",
           "fa_bwd_mod_workspace_size", "fa_rope",
           "fa_rope_append", "fa_fwd_tree_workspace_size", "fa_fwd_tree", "fa_strerror", "fa_version")

_lock = threading.Lock()
_lib = None


class FAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: status {status} ({strerror(status)})")


def lib() -> ctypes.CDLL:
    """Load libfa.so (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with exact_attention_23_gb300.build.build()")
            L = ctypes.CDLL(LIB_PATH)
            vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
            L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp]
            L.fa_fwd.restype = i
            L.fa_fwd_ex.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp,
                                    ctypes.c_ulonglong, ctypes.c_uint, vp]
            L.fa_fwd_ex.restype = i
            sz = ctypes.c_size_t
            L.fa_fwd_fp8.argtypes = [vp] * 5 + [f, f, i, i, i, i, i, f, vp]
            L.fa_fwd_host_workspace_size.argtypes = [i, i, i, i, i]
            L.fa_fwd_host_workspace_size.restype = sz
            L.fa_fwd_host.argtypes = [vp] * 5 + [i, i, i, i, i, f, i, vp, sz, vp]
            L.fa_fwd_host.restype = i
            L.fa_fwd_fp8.restype = i
            L.fa_fwd_kv_workspace_size.argtypes = [i, i, i, i, i, i]
            L.fa_fwd_kv_workspace_size.restype = sz
            L.fa_fwd_kv.argtypes = [vp] * 5 + [i, i, i, i, i, i, f, i, vp, sz, vp]
            L.fa_fwd_kv.restype = i
            L.fa_fwd_block_sparse.argtypes = [vp] * 6 + [i, i, i, i, i, i, f, vp]
            L.fa_fwd_block_sparse.restype = i
            L.fa_bwd_workspace_size.argtypes = [i, i, i, i]
            L.fa_bwd_workspace_size.restype = sz
            L.fa_bwd.argtypes = [vp] * 10 + [sz, i, i, i, i, i, f, vp]
            L.fa_bwd.restype = i
            L.fa_bwd_ex.argtypes = [vp] * 10 + [sz, i, i, i, i, i, f, vp, ctypes.c_ulonglong,
                                                ctypes.c_uint, vp]
            L.fa_bwd_ex.restype = i
            L.fa_bwd_noalloc.argtypes = [vp] * 9 + [i, i, i, i, i, f, vp]
            L.fa_bwd_noalloc.restype = i
            L.fa_visible_size.argtypes = [i, i]
            L.fa_visible_size.restype = sz
            L.fa_visible.argtypes = [vp, vp, i, i, vp, sz, i, i, vp]
            L.fa_visible.restype = i
            ull, ll = ctypes.c_ulonglong, ctypes.c_longlong
            L.fa_fwd_mod.argtypes = [vp] * 7 + [i, f, vp, i, i, i, i, i, f, vp, ull, vp]
            L.fa_fwd_mod.restype = i
            L.fa_bwd_mod.argtypes = [vp] * 11 + [sz, vp, i, f, vp, i, i, i, i, i, f, vp, ull, vp]
            L.fa_bwd_mod.restype = i
            L.fa_bwd_mod_workspace_size.argtypes = [i] * 5
            L.fa_bwd_mod_workspace_size.restype = sz
            src = [vp, ll, ll, ll]
            L.fa_rope.argtypes = src + [vp] + src + [vp, vp, i, vp, i, i, i, f, i, i, i, i, i, vp]
            L.fa_rope.restype = i
            L.fa_rope_append.argtypes = (src + [vp] + src + src + [vp, vp, vp, vp, i, vp, i, i, f]
                                         + [i] * 6 + [vp])
            L.fa_rope_append.restype = i
            L.fa_fwd_tree_workspace_size.argtypes = [i] * 6
            L.fa_fwd_tree_workspace_size.restype = sz
            L.fa_fwd_tree.argtypes = ([vp] * 7 + [i, vp, i, f, vp] + [i] * 6 + [f, vp, sz, vp, ull, vp])
            L.fa_fwd_tree.restype = i
            L.fa_strerror.argtypes = [i]
            L.fa_strerror.restype = ctypes.c_char_p
            L.fa_version.argtypes = []
            L.fa_version.restype = ctypes.c_char_p
            _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().fa_strerror(int(status)).decode()


def version() -> str:
    return lib().fa_version().decode()


def fa_fwd(q, k, v, o, lse, B, H, T, d, causal, scale, stream) -> int:
    """Raw call: integer addresses in, status out."""
    return lib().fa_fwd(q, k, v, o, lse, B, H, T, d, int(bool(causal)), float(scale), stream)


def fa_fwd_ex(q, k, v, o, lse, B, H, T, d, causal, scale, status, timeout_ns, flags,
              stream) -> int:
    return lib().fa_fwd_ex(q, k, v, o, lse, B, H, T, d, int(bool(causal)), float(scale),
                           status, int(timeout_ns), int(flags), stream)


def fa_bwd_workspace_size(B, H, T, d) -> int:
    return int(lib().fa_bwd_workspace_size(B, H, T, d))


def fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, workspace, workspace_bytes, B, H, T, d, causal,
           scale, stream) -> int:
    return lib().fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, workspace, int(workspace_bytes), B,
                        H, T, d, int(bool(causal)), float(scale), stream)


def fa_bwd_ex(q, k, v, o, dout, lse, dq, dk, dv, workspace, workspace_bytes, B, H, T, d,
              causal, scale, status, timeout_ns, flags, stream) -> int:
    return lib().fa_bwd_ex(q, k, v, o, dout, lse, dq, dk, dv, workspace, int(workspace_bytes),
                           B, H, T, d, int(bool(causal)), float(scale), status,
                           int(timeout_ns), int(flags), stream)


def fa_bwd_noalloc(q, k, v, o, dout, lse, dq, dk, dv, B, H, T, d, causal, scale, stream) -> int:
    return lib().fa_bwd_noalloc(q, k, v, o, dout, lse, dq, dk, dv, B, H, T, d,
                                int(bool(causal)), float(scale), stream)


def fa_fwd_kv_workspace_size(B, H, Tq, Tk, d, n_splits) -> int:
    return int(lib().fa_fwd_kv_workspace_size(B, H, Tq, Tk, d, n_splits))


def fa_fwd_kv(q, k, v, o, lse, B, H, Tq, Tk, d, causal, scale, n_splits, workspace,
              workspace_bytes, stream) -> int:
    return lib().fa_fwd_kv(q, k, v, o, lse, B, H, Tq, Tk, d, int(bool(causal)), float(scale),
                           int(n_splits), workspace, int(workspace_bytes), stream)


def fa_fwd_block_sparse(q, k, v, o, lse, block_mask, mask_heads, B, H, T, d, causal, scale,
                        stream) -> int:
    return lib().fa_fwd_block_sparse(q, k, v, o, lse, block_mask, int(mask_heads), B, H, T, d,
                                     int(bool(causal)), float(scale), stream)


def fa_fwd_fp8(q8, k8, v, o, lse, q_scale, k_scale, B, H, T, d, causal, scale, stream) -> int:
    return lib().fa_fwd_fp8(q8, k8, v, o, lse, float(q_scale), float(k_scale), B, H, T, d,
                            int(bool(causal)), float(scale), stream)


def fa_fwd_host_workspace_size(B, H, T, d, heads_per_chunk=0) -> int:
    return int(lib().fa_fwd_host_workspace_size(B, H, T, d, heads_per_chunk))


def fa_fwd_host(q, k, v, o, lse, B, H, T, d, causal, scale, heads_per_chunk, ws, ws_bytes,
                stream) -> int:
    return lib().fa_fwd_host(q, k, v, o, lse, B, H, T, d, int(bool(causal)), float(scale),
                             heads_per_chunk, ws, ws_bytes, stream)


def fa_visible_size(B, T) -> int:
    return int(lib().fa_visible_size(B, T))


def fa_visible(doc_ids, prefix_len, prefix_per_token, causal, visible, visible_bytes, B, T,
               stream) -> int:
    return lib().fa_visible(doc_ids, prefix_len, int(prefix_per_token), int(bool(causal)), visible,
                            int(visible_bytes), B, T, stream)


def fa_fwd_mod(q, k, v, o, lse, rest, visible, causal, softcap, slopes, B, H, Hkv, T, d, scale,
               status, timeout_ns, stream) -> int:
    return lib().fa_fwd_mod(q, k, v, o, lse, rest, visible, int(bool(causal)), float(softcap), slopes, B,
                            H, Hkv, T, d, float(scale), status, int(timeout_ns), stream)


def fa_bwd_mod(q, k, v, o, dout, lse, rest, dq, dk, dv, workspace, workspace_bytes, visible, causal,
               softcap, slopes, B, H, Hkv, T, d, scale, status, timeout_ns, stream) -> int:
    return lib().fa_bwd_mod(q, k, v, o, dout, lse, rest, dq, dk, dv, workspace, int(workspace_bytes),
                            visible, int(bool(causal)), float(softcap), slopes, B, H, Hkv, T, d,
                            float(scale), status, int(timeout_ns), stream)


def fa_bwd_mod_workspace_size(B, H, Hkv, T, d) -> int:
    return int(lib().fa_bwd_mod_workspace_size(B, H, Hkv, T, d))


def fa_rope(q, q_strides, q_out, k, k_strides, k_out, positions, positions_per_batch, inv_freq,
            rot_dim, interleaved, inverse, mscale, B, H, Hkv, T, d, stream) -> int:
    """q_strides and k_strides: (batch, head, token), in elements."""
    return lib().fa_rope(q, *q_strides, q_out, k, *k_strides, k_out, positions,
                         int(positions_per_batch), inv_freq, rot_dim, int(interleaved),
                         int(inverse), float(mscale), B, H, Hkv, T, d, stream)


def fa_rope_append(q, q_strides, q_out, k, k_strides, v, v_strides, k_cache, v_cache, ctx_len,
                   positions, positions_per_batch, inv_freq, rot_dim, interleaved, mscale, B, H,
                   Hkv, Tq, Tmax, d, stream) -> int:
    return lib().fa_rope_append(q, *q_strides, q_out, k, *k_strides, v, *v_strides, k_cache,
                                v_cache, ctx_len, positions, int(positions_per_batch), inv_freq,
                                rot_dim, int(interleaved), float(mscale), B, H, Hkv, Tq, Tmax, d,
                                stream)


def fa_fwd_tree_workspace_size(B, H, Hkv, Tq, Tmax, d) -> int:
    return int(lib().fa_fwd_tree_workspace_size(B, H, Hkv, Tq, Tmax, d))


def fa_fwd_tree(q, k_cache, v_cache, o, lse, ctx_len, tree, tree_per_batch, depths,
                depths_per_batch, softcap, slopes, B, H, Hkv, Tq, Tmax, d, scale, workspace,
                workspace_bytes, status, timeout_ns, stream) -> int:
    return lib().fa_fwd_tree(q, k_cache, v_cache, o, lse, ctx_len, tree, int(tree_per_batch), depths,
                             int(depths_per_batch), float(softcap), slopes, B, H, Hkv, Tq, Tmax, d,
                             float(scale), workspace, int(workspace_bytes), status, int(timeout_ns),
                             stream)

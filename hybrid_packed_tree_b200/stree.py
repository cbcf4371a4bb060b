"""Thin ctypes binding of ``libstree.so`` (the C ABI declared in include/stree.h).

Argument marshalling only: shapes are read from the torch tensors, pointers are
passed as they are, and every step of the scan runs in the library's CUDA
kernels.  Importing this module loads the library and raises ImportError when it
has not been built (``python -m hybrid_packed_tree_b200.build``); there is no
fallback for a kernel.  The argument check in C++ is an addition to the one here and is
taken when it has been compiled for the running torch and Python.

The functions carry the C names.  Tensors must be contiguous CUDA tensors in the
layouts of the header: x [b,T,H,P], dt [b,T,H], A/D [H] fp32, B/C [b,T,G,N],
h0/h_new [b,H,P,N] fp32, y like x, parent [b,T] int32, path [b,maxlen] int32,
path_len [b] int32.  ``stream`` defaults to torch's current stream.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import warnings

import torch

from .build import LIB, bind_path

if not os.path.exists(LIB):
    raise ImportError(f"libstree.so is not built ({LIB}); run `python -m hybrid_packed_tree_b200.build`")

_lib = ctypes.CDLL(LIB)

STREE_OK = 0
STATUS_NAMES = {
    0: "STREE_OK", 1: "STREE_ERR_INVALID_ARG", 2: "STREE_ERR_UNSUPPORTED", 3: "STREE_ERR_BAD_TREE",
    4: "STREE_ERR_BAD_PATH", 5: "STREE_ERR_MISALIGNED", 6: "STREE_ERR_CUDA", 7: "STREE_ERR_TIMEOUT",
    8: "STREE_ERR_NO_TREE", 9: "STREE_ERR_BAD_SEQ", 10: "STREE_ERR_BAD_PAGE",
}
STREE_F32, STREE_BF16, STREE_E4M3 = 0, 1, 2
KERNELS = {"auto": 0, "simt": 1, "tc": 2, "small": 3}

# Every exported symbol of include/stree.h.
EXPORTS = (
    "stree_ctx_create", "stree_ctx_destroy", "stree_ctx_set_kernel", "stree_ctx_launch_count",
    "stree_ctx_last_kernel", "stree_ctx_set_wait_limit", "stree_ctx_set_test_fault", "stree_set_wait_hook",
    "stree_build_tree",
    "stree_tree_scan", "stree_commit", "stree_tree_scan_commit", "stree_tree_scan_commit_noalloc",
    "stree_resolve_path", "stree_unrolled_scan", "stree_accept_greedy", "stree_accept_sampling",
    "stree_gdn_tree_scan_commit", "stree_tree_attention", "stree_tree_attention_workspace_size",
    "stree_linear_prompt", "stree_linear_prompt_workspace_size", "stree_linear_step", "stree_prompt_attention",
    "stree_paged_attention", "stree_paged_attention_workspace_size", "stree_cache_write", "stree_cache_commit",
    "stree_cache_read",
    "stree_sync_check", "stree_status_string", "stree_version",
)

_vp, _i, _ip = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_int32)
_lib.stree_ctx_create.argtypes = [ctypes.POINTER(_vp)]
_lib.stree_ctx_destroy.argtypes = [_vp]
_lib.stree_ctx_set_kernel.argtypes = [_vp, _i]
_lib.stree_ctx_launch_count.argtypes = [_vp, ctypes.POINTER(ctypes.c_int64)]
_lib.stree_ctx_last_kernel.argtypes = [_vp, ctypes.POINTER(ctypes.c_int)]
_lib.stree_ctx_set_wait_limit.argtypes = [_vp, ctypes.c_uint64]
_lib.stree_ctx_set_test_fault.argtypes = [_vp, _i]
_lib.stree_set_wait_hook.argtypes = [_vp]
_lib.stree_build_tree.argtypes = [_vp, _vp, _i, _i, _vp, _vp, _vp]
_lib.stree_tree_scan.argtypes = [_vp] * 9 + [_i] * 7 + [_vp, _vp]
_lib.stree_commit.argtypes = [_vp, _vp, _vp, _i, _vp, _vp]
_lib.stree_tree_scan_commit.argtypes = [_vp] * 9 + [_i] * 7 + [_vp, _vp, _i, _vp, _vp, _vp]
_lib.stree_tree_scan_commit_noalloc.argtypes = [_vp] * 8 + [_i] * 7 + [_vp, _vp, _i, _vp, _vp, _vp, _vp]
_lib.stree_resolve_path.argtypes = [_vp, _vp, _vp, _i, _vp, _vp]
_lib.stree_unrolled_scan.argtypes = [_vp] * 9 + [_i] * 9 + [_vp, _vp, _vp, _vp]
_lib.stree_accept_greedy.argtypes = [_vp, _i, _i, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.stree_accept_sampling.argtypes = [_vp, _vp, _i, _i, _vp, _vp, _i, _i, ctypes.c_float, _vp, _vp, _i, _vp,
                                        _vp, _vp, _vp, _vp]
_lib.stree_gdn_tree_scan_commit.argtypes = [_vp] * 8 + [_i] * 7 + [_vp, _vp, _i, _vp, _vp, _vp, _vp]
_lib.stree_tree_attention.argtypes = [_vp] * 7 + [_i] * 6 + [ctypes.c_float, _i, _vp, _vp, ctypes.c_size_t, _vp, _vp]
_lib.stree_tree_attention_workspace_size.argtypes = [_i] * 6 + [ctypes.POINTER(ctypes.c_size_t)]
_lib.stree_linear_prompt.argtypes = [_vp] * 8 + [_i] * 7 + [_vp, _vp, _vp, ctypes.c_size_t, _vp, _vp]
_lib.stree_linear_prompt_workspace_size.argtypes = [_i] * 7 + [ctypes.POINTER(ctypes.c_size_t)]
_lib.stree_linear_step.argtypes = [_vp] * 7 + [_i] * 6 + [_vp, _vp, _vp]
_lib.stree_prompt_attention.argtypes = [_vp] * 4 + [_i] * 5 + [ctypes.c_float, _i, _vp, _vp, _vp]
_lib.stree_paged_attention.argtypes = [_vp] * 7 + [_i] * 7 + [ctypes.c_float, _i, _i, _vp, _vp, ctypes.c_size_t, _vp,
                                                                _vp]
_lib.stree_paged_attention_workspace_size.argtypes = [_i] * 3 + [ctypes.POINTER(ctypes.c_size_t)]
_lib.stree_cache_write.argtypes = [_vp] * 5 + [_i] * 9 + [_vp] * 6
_lib.stree_cache_commit.argtypes = [_vp] * 4 + [_i, _vp, _vp] + [_i] * 9 + [_vp] * 6
_lib.stree_cache_read.argtypes = [_vp] * 6 + [_i] * 9 + [_vp] * 4
_lib.stree_sync_check.argtypes = [_vp, _vp, _ip]
_lib.stree_status_string.argtypes = [_i]
_lib.stree_status_string.restype = ctypes.c_char_p
_lib.stree_version.argtypes = []
for _name in EXPORTS:
    if _name not in ("stree_status_string",):
        getattr(_lib, _name).restype = ctypes.c_int


class StreeError(RuntimeError):
    def __init__(self, status: int, where: str, info=None):
        self.status = int(status)
        self.info = info
        msg = f"{where}: {STATUS_NAMES.get(status, status)} ({stree_status_string(status)})"
        if info is not None:
            msg += f" info={list(info)}"
        super().__init__(msg)


def _check(st: int, where: str):
    if st != STREE_OK:
        raise StreeError(st, where)


def stree_status_string(status: int) -> str:
    return _lib.stree_status_string(int(status)).decode()


def stree_version() -> int:
    return int(_lib.stree_version())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr(t, name, dtypes=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    return ctypes.c_void_p(t.data_ptr())


def _io_dtype(x):
    if x.dtype == torch.bfloat16:
        return STREE_BF16
    if x.dtype == torch.float32:
        return STREE_F32
    raise TypeError(f"x has dtype {x.dtype}; fp32 and bf16 are supported")


class Ctx:
    """Owns one ``stree_ctx``; closed by ``stree_ctx_destroy`` (or garbage collection)."""

    def __init__(self):
        h = ctypes.c_void_p()
        _check(_lib.stree_ctx_create(ctypes.byref(h)), "stree_ctx_create")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None):
            _lib.stree_ctx_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def stree_ctx_create() -> Ctx:
    return Ctx()


def stree_ctx_destroy(ctx: Ctx):
    ctx.close()


def stree_ctx_set_kernel(ctx: Ctx, kernel="auto"):
    k = KERNELS[kernel] if isinstance(kernel, str) else int(kernel)
    _check(_lib.stree_ctx_set_kernel(ctx.handle, k), "stree_ctx_set_kernel")


def stree_ctx_launch_count(ctx: Ctx) -> int:
    n = ctypes.c_int64(0)
    _check(_lib.stree_ctx_launch_count(ctx.handle, ctypes.byref(n)), "stree_ctx_launch_count")
    return int(n.value)


def stree_ctx_last_kernel(ctx: Ctx) -> str:
    """Name ("simt", "tc" or "small") of the kernel that ran the last scan; "auto" before any."""
    k = ctypes.c_int(0)
    _check(_lib.stree_ctx_last_kernel(ctx.handle, ctypes.byref(k)), "stree_ctx_last_kernel")
    return {v: n for n, v in KERNELS.items()}[int(k.value)]


def stree_ctx_set_wait_limit(ctx: Ctx, ns: int = 0):
    """Bounded-wait limit of the tensor-core kernel in ns (0: the default, about 1 s)."""
    _check(_lib.stree_ctx_set_wait_limit(ctx.handle, int(ns)), "stree_ctx_set_wait_limit")


def stree_ctx_set_test_fault(ctx: Ctx, fault: int = 0):
    """Failure-path test hook: 1 makes a bounded wait of the tensor-core kernel run out."""
    _check(_lib.stree_ctx_set_test_fault(ctx.handle, int(fault)), "stree_ctx_set_test_fault")


class _WaitHook(ctypes.Structure):
    _fields_ = [("wait_ns", ctypes.c_uint64), ("fault", ctypes.c_int)]


def stree_set_wait_hook(wait_ns: int = 0, fault: int = 0):
    """Bounded-wait limit in ns (0: about 1 s) of the calls without a context that hand work between
    warp roles, for later calls of this thread; fault=1, a test hook, makes one of their waits run out."""
    if not 0 <= int(wait_ns) < 1 << 64:
        raise ValueError("wait_ns must be a number of nanoseconds")
    hook = _WaitHook(int(wait_ns), int(fault))
    _check(_lib.stree_set_wait_hook(ctypes.byref(hook)), "stree_set_wait_hook")


def stree_build_tree(ctx: Ctx, parent, anc_out=None, depth_out=None, stream=None):
    batch, T = parent.shape
    _check(_lib.stree_build_tree(ctx.handle, _ptr(parent, "parent", (torch.int32,)), T, batch,
                                 _ptr(anc_out, "anc_out", (torch.int32,)),
                                 _ptr(depth_out, "depth_out", (torch.int32,)), _stream(stream)),
           "stree_build_tree")


def _scan_ptrs(x, dt, A, B, C, D, h0, y):
    io = (x.dtype,)
    return [_ptr(x, "x", (torch.float32, torch.bfloat16)), _ptr(dt, "dt", io), _ptr(A, "A", (torch.float32,)),
            _ptr(B, "B", io), _ptr(C, "C", io), _ptr(D, "D", (torch.float32,)),
            _ptr(h0, "h0", (torch.float32,))], _ptr(y, "y", io)


def _dims(x, B):
    batch, T, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    return [T, batch, H, P, N, G]


def stree_tree_scan(ctx: Ctx, x, dt, A, B, C, D, h0, parent, y, stream=None):
    """y <- packed tree scan.  parent=None reuses the context's current tree."""
    ins, yp = _scan_ptrs(x, dt, A, B, C, D, h0, y)
    st = _lib.stree_tree_scan(ctx.handle, *ins, _ptr(parent, "parent", (torch.int32,)),
                              *_dims(x, B), _io_dtype(x), yp, _stream(stream))
    _check(st, "stree_tree_scan")
    return y


def stree_commit(ctx: Ctx, path, path_len, h_new, stream=None):
    """h_new <- activation replay of the accepted paths over the last scan's inputs."""
    st = _lib.stree_commit(ctx.handle, _ptr(path, "path", (torch.int32,)),
                           _ptr(path_len, "path_len", (torch.int32,)), path.shape[1],
                           _ptr(h_new, "h_new", (torch.float32,)), _stream(stream))
    _check(st, "stree_commit")
    return h_new


def stree_tree_scan_commit(ctx: Ctx, x, dt, A, B, C, D, h0, parent, path, path_len, y, h_new, stream=None):
    """(y, h_new) <- fused scan + commit (h0 read once)."""
    ins, yp = _scan_ptrs(x, dt, A, B, C, D, h0, y)
    st = _lib.stree_tree_scan_commit(ctx.handle, *ins, _ptr(parent, "parent", (torch.int32,)),
                                     *_dims(x, B), _io_dtype(x),
                                     _ptr(path, "path", (torch.int32,)),
                                     _ptr(path_len, "path_len", (torch.int32,)), path.shape[1],
                                     yp, _ptr(h_new, "h_new", (torch.float32,)), _stream(stream))
    _check(st, "stree_tree_scan_commit")
    return y, h_new


def stree_tree_scan_commit_noalloc(x, dt, A, B, C, D, h0, parent, path, path_len, y, h_new, err_out=None,
                                   stream=None):
    """(y, h_new) <- fused scan + commit with no context and no allocation.

    Scratch comes from the library's fixed device array; err_out (device int32[4])
    receives this call's error word.  Calls on one device must not overlap.
    """
    ins, yp = _scan_ptrs(x, dt, A, B, C, D, h0, y)
    st = _lib.stree_tree_scan_commit_noalloc(*ins, _ptr(parent, "parent", (torch.int32,)), *_dims(x, B),
                                             _io_dtype(x), _ptr(path, "path", (torch.int32,)),
                                             _ptr(path_len, "path_len", (torch.int32,)), path.shape[1], yp,
                                             _ptr(h_new, "h_new", (torch.float32,)),
                                             _ptr(err_out, "err_out", (torch.int32,)), _stream(stream))
    _check(st, "stree_tree_scan_commit_noalloc")
    return y, h_new


def stree_unrolled_scan(x, dt, A, B, C, D, h0, paths, path_len, y_paths, h_paths, err_out=None, stream=None):
    """(y_paths, h_paths) <- every path scanned as its own sequence (the unrolled-tree baseline).

    paths [b, n_paths, max_depth] int32, path_len [b, n_paths] int32,
    y_paths [b, n_paths, max_depth, H, P] in x's dtype, h_paths [b, n_paths, H, P, N] fp32.
    """
    ins, yp = _scan_ptrs(x, dt, A, B, C, D, h0, y_paths)
    batch, T, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    st = _lib.stree_unrolled_scan(*ins[:7], _ptr(paths, "paths", (torch.int32,)),
                                  _ptr(path_len, "path_len", (torch.int32,)), T, batch, paths.shape[1],
                                  paths.shape[2], H, P, N, G, _io_dtype(x), yp,
                                  _ptr(h_paths, "h_paths", (torch.float32,)),
                                  _ptr(err_out, "err_out", (torch.int32,)), _stream(stream))
    _check(st, "stree_unrolled_scan")
    return y_paths, h_paths


def stree_accept_greedy(logits, draft_tokens, parent, pred, accepted_path, path_len, bonus_token, err_out=None,
                        stream=None):
    """Greedy tree verification: (pred, accepted_path, path_len, bonus_token) from the
    target's logits [b, T, V] (fp32 or bf16) and the draft tokens [b, T]."""
    batch, T, V = logits.shape
    st = _lib.stree_accept_greedy(_ptr(logits, "logits", (torch.float32, torch.bfloat16)), _io_dtype(logits), V,
                                  _ptr(draft_tokens, "draft_tokens", (torch.int32,)),
                                  _ptr(parent, "parent", (torch.int32,)), T, batch, accepted_path.shape[1],
                                  _ptr(pred, "pred", (torch.int32,)), _ptr(accepted_path, "accepted_path", (torch.int32,)),
                                  _ptr(path_len, "path_len", (torch.int32,)),
                                  _ptr(bonus_token, "bonus_token", (torch.int32,)),
                                  _ptr(err_out, "err_out", (torch.int32,)), _stream(stream))
    _check(st, "stree_accept_greedy")
    return pred, accepted_path, path_len, bonus_token


def stree_accept_sampling(target_logits, draft_logits, draft_tokens, parent, temperature, u_accept, u_bonus,
                          accepted_path, path_len, bonus_token, err_out=None, stream=None):
    """Stochastic tree verification by multi-step speculative sampling: (accepted_path,
    path_len, bonus_token) from the target's and the draft's logits [b, T, V] (fp32 or
    bf16, same dtype), the draft tokens [b, T] and the uniforms u_accept [b, T] and
    u_bonus [b] (fp32)."""
    batch, T, V = target_logits.shape
    if draft_logits.shape != target_logits.shape or draft_logits.dtype != target_logits.dtype:
        raise ValueError("draft_logits must match target_logits in shape and dtype")
    st = _lib.stree_accept_sampling(_ptr(target_logits, "target_logits", (torch.float32, torch.bfloat16)),
                                    _ptr(draft_logits, "draft_logits", (target_logits.dtype,)),
                                    _io_dtype(target_logits), V, _ptr(draft_tokens, "draft_tokens", (torch.int32,)),
                                    _ptr(parent, "parent", (torch.int32,)), T, batch, float(temperature),
                                    _ptr(u_accept, "u_accept", (torch.float32,)),
                                    _ptr(u_bonus, "u_bonus", (torch.float32,)), accepted_path.shape[1],
                                    _ptr(accepted_path, "accepted_path", (torch.int32,)),
                                    _ptr(path_len, "path_len", (torch.int32,)),
                                    _ptr(bonus_token, "bonus_token", (torch.int32,)),
                                    _ptr(err_out, "err_out", (torch.int32,)), _stream(stream))
    _check(st, "stree_accept_sampling")
    return accepted_path, path_len, bonus_token


def stree_gdn_tree_scan_commit(q, k, v, alpha, beta, S0, parent, o, path=None, path_len=None, S_new=None,
                               err_out=None, stream=None, erase=None):
    """Gated delta rule over the packed tree: o [b, T, Hv, dv] for every node and, when
    path / path_len / S_new are given, the accepted path's state S_new [b, Hv, dv, dk].
    q, k [b, T, Hk, dk] and v [b, T, Hv, dv] in one dtype (fp32 or bf16); alpha, beta
    [b, T, Hv] and S0 fp32; erase [b, T, Hv] fp32 (None: erase = beta; zeros: gated
    linear attention)."""
    batch, T, Hk, dk = k.shape
    Hv, dv = v.shape[2], v.shape[3]
    io = (v.dtype,)
    st = _lib.stree_gdn_tree_scan_commit(
        _ptr(q, "q", io), _ptr(k, "k", io), _ptr(v, "v", (torch.float32, torch.bfloat16)),
        _ptr(alpha, "alpha", (torch.float32,)), _ptr(beta, "beta", (torch.float32,)),
        _ptr(erase, "erase", (torch.float32,)), _ptr(S0, "S0", (torch.float32,)), _ptr(parent, "parent", (torch.int32,)), T, batch, Hv, Hk, dk, dv,
        _io_dtype(v), _ptr(path, "path", (torch.int32,)), _ptr(path_len, "path_len", (torch.int32,)),
        path.shape[1] if path is not None else 0, _ptr(o, "o", io), _ptr(S_new, "S_new", (torch.float32,)),
        _ptr(err_out, "err_out", (torch.int32,)), _stream(stream))
    _check(st, "stree_gdn_tree_scan_commit")
    return o, S_new


def stree_tree_attention_workspace_size(n_nodes, batch, ctx_cap, heads_q, heads_kv, head_dim=128) -> int:
    """Bytes of the workspace stree_tree_attention splits into on the current device (0: no split)."""
    n = ctypes.c_size_t(0)
    _check(_lib.stree_tree_attention_workspace_size(int(n_nodes), int(batch), int(ctx_cap), int(heads_q),
                                                    int(heads_kv), int(head_dim), ctypes.byref(n)),
           "stree_tree_attention_workspace_size")
    return int(n.value)


def stree_tree_attention(q, k_ctx, v_ctx, k_tree, v_tree, ctx_len, parent, o, scale, err_out, workspace=None,
                         stream=None):
    """Tree-masked attention: o [b, T, Hq, 128] (bf16) from q [b, T, Hq, 128], the
    context cache k_ctx / v_ctx [b, S, Hkv, 128] (S may be 0), the tree's own k_tree /
    v_tree [b, T, Hkv, 128], ctx_len [b] and parent [b, T].  workspace: a device
    uint8 tensor of stree_tree_attention_workspace_size() bytes, or None (no split)."""
    batch, T, Hq, d = q.shape
    S, Hkv = k_ctx.shape[1], k_ctx.shape[2]
    bf = (torch.bfloat16,)
    ws = _ptr(workspace, "workspace", (torch.uint8,)) if workspace is not None else None
    ws_bytes = workspace.numel() if workspace is not None else 0
    st = _lib.stree_tree_attention(_ptr(q, "q", bf), _ptr(k_ctx, "k_ctx", bf) if S else None,
                                   _ptr(v_ctx, "v_ctx", bf) if S else None, _ptr(k_tree, "k_tree", bf),
                                   _ptr(v_tree, "v_tree", bf), _ptr(ctx_len, "ctx_len", (torch.int32,)),
                                   _ptr(parent, "parent", (torch.int32,)), T, batch, S, Hq, Hkv, d, float(scale),
                                   STREE_BF16, _ptr(o, "o", bf), ws, ws_bytes,
                                   _ptr(err_out, "err_out", (torch.int32,)), _stream(stream))
    _check(st, "stree_tree_attention")
    return o


# ---------------------------------------------------------------- prompts, single tokens, the paged cache
#
# A decode step makes several of these calls per layer and token, so their tensors are checked in
# C++ (csrc/bind.cpp, where it has been compiled) and their pointers are plain integers.

_F32, _BF16, _I32, _U8, _E4M3 = torch.float32, torch.bfloat16, torch.int32, torch.uint8, torch.float8_e4m3fn
_IO = {torch.float32: STREE_F32, torch.bfloat16: STREE_BF16}


def _refuse(t, name, shape, dtype, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    raise ValueError(f"{name} must be contiguous")


# _arg(t, name, shape, dtype, dev): the pointer of a tensor of exactly this shape and dtype, contiguous, on
# CUDA device `dev` (_opt: or None); otherwise _refuse says what is wrong.  Asked property by property in
# Python, as here, a single-token call cost 9.4 us on the host, by csrc/bind.cpp 6.5.
def _arg(t, name, shape, dtype, dev):
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_cuda and t.get_device() == dev and
            t.layout is torch.strided and t.is_contiguous()):
        return t.data_ptr()
    _refuse(t, name, shape, dtype, dev)


def _opt(t, name, shape, dtype, dev):
    return None if t is None else _arg(t, name, shape, dtype, dev)


def _load_bind():
    """The check that was compiled for this torch and this Python, or None."""
    path = bind_path()
    if not os.path.exists(path):
        return None
    name = __package__ + "._bind"
    loader = importlib.machinery.ExtensionFileLoader(name, path)
    try:
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader(name, loader))
        loader.exec_module(module)
    except ImportError as e:
        warnings.warn(f"{path} does not load ({e}); arguments are checked in Python")
        return None
    module.on_refusal(_refuse)
    return module


_bind = _load_bind()
if _bind is not None:
    _arg, _opt = _bind.arg, _bind.opt


def _call(where, fn, dev, stream, *args):
    """Calls a library function on device `dev`, on that device's current stream when none is given."""
    if dev == torch._C._cuda_getDevice():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if st != STREE_OK:
        raise StreeError(st, where)


def _scratch(workspace, dev):
    if workspace is None:
        return None, 0
    n = workspace.numel()
    return _arg(workspace, "workspace", workspace.shape, _U8, dev), n


def stree_linear_prompt_workspace_size(batch, total, heads_v, heads_k, dk, dv, dtype=torch.bfloat16) -> int:
    """Bytes of the workspace in which stree_linear_prompt splits long sequences on the current device (0: no split)."""
    n = ctypes.c_size_t(0)
    _check(_lib.stree_linear_prompt_workspace_size(int(batch), int(total), int(heads_v), int(heads_k), int(dk), int(dv),
                                                   _IO.get(dtype, -1), ctypes.byref(n)),
           "stree_linear_prompt_workspace_size")
    return int(n.value)


def stree_linear_prompt(q, k, v, alpha, beta, cu_seqlens, o, S0=None, S_new=None, skip=None, err_out=None,
                        workspace=None, stream=None):
    """Linear attention with a decay for each head over packed prompts: o [total, Hv, dv] and, when
    S_new is given, the states [b, Hv, dv, dk] after the last tokens.  q, k [total, Hk, dk] and v in
    one dtype (fp32 or bf16); alpha, beta [total, Hv] fp32 (beta None: ones); S0 fp32 (None: zeros);
    skip [Hv] fp32 or None; cu_seqlens [b + 1] int32.  workspace: a device uint8 tensor of
    stree_linear_prompt_workspace_size() bytes, or None (long sequences are not split)."""
    total, Hk, dk = k.shape
    _, Hv, dv = v.shape
    batch, io, dev = cu_seqlens.shape[0] - 1, v.dtype, v.get_device()
    rows, keys, gates, state = (total, Hv, dv), (total, Hk, dk), (total, Hv), (batch, Hv, dv, dk)
    ws, ws_bytes = _scratch(workspace, dev)
    _call("stree_linear_prompt", _lib.stree_linear_prompt, dev, stream, _arg(q, "q", keys, io, dev),
          _arg(k, "k", keys, io, dev), _arg(v, "v", rows, io, dev), _arg(alpha, "alpha", gates, _F32, dev),
          _opt(beta, "beta", gates, _F32, dev), _opt(skip, "skip", (Hv,), _F32, dev), _opt(S0, "S0", state, _F32, dev),
          _arg(cu_seqlens, "cu_seqlens", (batch + 1,), _I32, dev), total, batch, Hv, Hk, dk, dv, _IO.get(io, -1),
          _arg(o, "o", rows, io, dev), _opt(S_new, "S_new", state, _F32, dev), ws, ws_bytes,
          _opt(err_out, "err_out", (4,), _I32, dev))
    return o, S_new


def stree_linear_step(q, k, v, alpha, beta, S0, o, S_new, skip=None, stream=None):
    """One token of stree_linear_prompt's recurrence for every sequence: (o [b, Hv, dv], S_new) from
    q, k [b, Hk, dk], v [b, Hv, dv], alpha, beta [b, Hv] (beta None: ones) and S0 (S_new may be S0)."""
    batch, Hk, dk = k.shape
    _, Hv, dv = v.shape
    io, dev = v.dtype, v.get_device()
    rows, keys, gates, state = (batch, Hv, dv), (batch, Hk, dk), (batch, Hv), (batch, Hv, dv, dk)
    _call("stree_linear_step", _lib.stree_linear_step, dev, stream, _arg(q, "q", keys, io, dev),
          _arg(k, "k", keys, io, dev), _arg(v, "v", rows, io, dev), _arg(alpha, "alpha", gates, _F32, dev),
          _opt(beta, "beta", gates, _F32, dev), _opt(skip, "skip", (Hv,), _F32, dev), _arg(S0, "S0", state, _F32, dev),
          batch, Hv, Hk, dk, dv, _IO.get(io, -1), _arg(o, "o", rows, io, dev), _arg(S_new, "S_new", state, _F32, dev))
    return o, S_new


def stree_prompt_attention(q, k, v, cu_seqlens, o, scale, err_out=None, stream=None):
    """Causal attention over packed prompts: o [total, Hq, 128] from q, k, v [total, H, 128] (bf16) and
    cu_seqlens [b + 1] int32."""
    total, Hq, d = q.shape
    Hkv = k.shape[1]
    batch, dev = cu_seqlens.shape[0] - 1, q.get_device()
    rows, keys = (total, Hq, d), (total, Hkv, d)
    _call("stree_prompt_attention", _lib.stree_prompt_attention, dev, stream, _arg(q, "q", rows, _BF16, dev),
          _arg(k, "k", keys, _BF16, dev), _arg(v, "v", keys, _BF16, dev),
          _arg(cu_seqlens, "cu_seqlens", (batch + 1,), _I32, dev), total, batch, Hq, Hkv, d, scale, STREE_BF16,
          _arg(o, "o", rows, _BF16, dev), _opt(err_out, "err_out", (4,), _I32, dev))
    return o


def _cache(k_pages, v_pages, page_table, k_scales, v_scales, batch, dev):
    """Pointers and sizes of a paged cache: (k, v, k scales, v scales, table), (heads, head dim, n_pages,
    page size, pages per sequence), its dtype code."""
    shape, pages = k_pages.shape, k_pages.dtype
    if len(shape) != 4 or page_table.dim() != 2:
        raise ValueError("k_pages is [n_pages, Hkv, page_size, 128] and page_table [batch, max_pages]")
    n_pages, Hkv, page, d = shape
    max_pages = page_table.shape[1]
    code = STREE_BF16
    if pages is _E4M3:
        code = STREE_E4M3
    elif pages is not _BF16:
        raise TypeError(f"k_pages has dtype {pages}, expected torch.bfloat16 or torch.float8_e4m3fn")
    if (k_scales is not None) != (code == STREE_E4M3) or (v_scales is not None) != (code == STREE_E4M3):
        raise ValueError("k_scales and v_scales go with float8_e4m3fn pages, and with them alone")
    return ((_arg(k_pages, "k_pages", shape, pages, dev), _arg(v_pages, "v_pages", shape, pages, dev),
             _opt(k_scales, "k_scales", (n_pages, Hkv, page), _U8, dev),
             _opt(v_scales, "v_scales", (n_pages, Hkv, page), _U8, dev),
             _arg(page_table, "page_table", (batch, max_pages), _I32, dev)), (Hkv, d, n_pages, page, max_pages), code)


def stree_paged_attention_workspace_size(heads_q, heads_kv, head_dim=128) -> int:
    """Bytes of stree_paged_attention's workspace on the current device (any batch and length)."""
    n = ctypes.c_size_t(0)
    _check(_lib.stree_paged_attention_workspace_size(int(heads_q), int(heads_kv), int(head_dim), ctypes.byref(n)),
           "stree_paged_attention_workspace_size")
    return int(n.value)


def stree_paged_attention(q, k_pages, v_pages, page_table, seq_len, o, scale, k_scales=None, v_scales=None,
                          err_out=None, workspace=None, stream=None):
    """One new token per sequence over its paged cache: o [b, Hq, 128] (bf16) from q [b, Hq, 128],
    pages [n, Hkv, page, 128] (bf16, or float8_e4m3fn with uint8 scales [n, Hkv, page]), page_table
    [b, max_pages] and seq_len [b] int32.  workspace: a device uint8 tensor of
    stree_paged_attention_workspace_size() bytes."""
    batch, Hq, d = q.shape
    dev = q.get_device()
    ptrs, sizes, code = _cache(k_pages, v_pages, page_table, k_scales, v_scales, batch, dev)
    rows = (batch, Hq, sizes[1])
    ws, ws_bytes = _scratch(workspace, dev)
    _call("stree_paged_attention", _lib.stree_paged_attention, dev, stream, _arg(q, "q", rows, _BF16, dev), *ptrs,
          _arg(seq_len, "seq_len", (batch,), _I32, dev), batch, Hq, *sizes, scale, STREE_BF16, code,
          _arg(o, "o", rows, _BF16, dev), ws, ws_bytes, _opt(err_out, "err_out", (4,), _I32, dev))
    return o


def stree_cache_write(k, v, cu_seqlens, start, page_table, k_pages, v_pages, k_scales=None, v_scales=None,
                      err_out=None, stream=None):
    """Writes packed new keys and values k, v [total, Hkv, 128] (bf16) into the pages, token i of
    sequence b at position start[b] + i; quantised as they are written when the pages are
    float8_e4m3fn (one power-of-two scale per row, in k_scales and v_scales)."""
    total, batch, dev = k.shape[0], start.shape[0], k.get_device()
    ptrs, sizes, code = _cache(k_pages, v_pages, page_table, k_scales, v_scales, batch, dev)
    rows = (total, sizes[0], sizes[1])
    _call("stree_cache_write", _lib.stree_cache_write, dev, stream, _arg(k, "k", rows, _BF16, dev),
          _arg(v, "v", rows, _BF16, dev), _arg(cu_seqlens, "cu_seqlens", (batch + 1,), _I32, dev),
          _arg(start, "start", (batch,), _I32, dev), ptrs[4], total, batch, *sizes, STREE_BF16, code, *ptrs[:4],
          _opt(err_out, "err_out", (4,), _I32, dev))
    return k_pages, v_pages


def stree_cache_commit(k_tree, v_tree, path, path_len, start, page_table, k_pages, v_pages, k_scales=None,
                       v_scales=None, err_out=None, stream=None):
    """Writes the accepted path of each tree into the pages: node path[b, i] of k_tree, v_tree
    [b, T, Hkv, 128] (bf16) at position start[b] + i, i < path_len[b]."""
    batch, T = k_tree.shape[:2]
    maxlen, dev = path.shape[1], k_tree.get_device()
    ptrs, sizes, code = _cache(k_pages, v_pages, page_table, k_scales, v_scales, batch, dev)
    rows = (batch, T, sizes[0], sizes[1])
    _call("stree_cache_commit", _lib.stree_cache_commit, dev, stream, _arg(k_tree, "k_tree", rows, _BF16, dev),
          _arg(v_tree, "v_tree", rows, _BF16, dev), _arg(path, "path", (batch, maxlen), _I32, dev),
          _arg(path_len, "path_len", (batch,), _I32, dev), maxlen, _arg(start, "start", (batch,), _I32, dev), ptrs[4], T,
          batch, *sizes, STREE_BF16, code, *ptrs[:4], _opt(err_out, "err_out", (4,), _I32, dev))
    return k_pages, v_pages


def stree_cache_read(k_pages, v_pages, page_table, seq_len, k_ctx, v_ctx, k_scales=None, v_scales=None, err_out=None,
                     stream=None):
    """Reads the first seq_len[b] positions of the pages back into the contiguous cache of
    stree_tree_attention, k_ctx, v_ctx [b, S, Hkv, 128] (bf16); later positions are untouched."""
    batch, S = k_ctx.shape[:2]
    dev = k_ctx.get_device()
    ptrs, sizes, code = _cache(k_pages, v_pages, page_table, k_scales, v_scales, batch, dev)
    rows = (batch, S, sizes[0], sizes[1])
    _call("stree_cache_read", _lib.stree_cache_read, dev, stream, *ptrs,
          _arg(seq_len, "seq_len", (batch,), _I32, dev), batch, S, *sizes, code, STREE_BF16,
          _arg(k_ctx, "k_ctx", rows, _BF16, dev), _arg(v_ctx, "v_ctx", rows, _BF16, dev),
          _opt(err_out, "err_out", (4,), _I32, dev))
    return k_ctx, v_ctx


def stree_resolve_path(ctx: Ctx, path, path_len, leaf_out, stream=None):
    st = _lib.stree_resolve_path(ctx.handle, _ptr(path, "path", (torch.int32,)),
                                 _ptr(path_len, "path_len", (torch.int32,)), path.shape[1],
                                 _ptr(leaf_out, "leaf_out", (torch.int32,)), _stream(stream))
    _check(st, "stree_resolve_path")
    return leaf_out


def stree_sync_check(ctx: Ctx, stream=None, raise_on_error: bool = True):
    """Synchronise, read and clear the device error word; returns (status, info[4])."""
    info = (ctypes.c_int32 * 4)()
    st = _lib.stree_sync_check(ctx.handle, _stream(stream), info)
    if st != STREE_OK and raise_on_error:
        raise StreeError(st, "stree_sync_check", list(info))
    return st, list(info)

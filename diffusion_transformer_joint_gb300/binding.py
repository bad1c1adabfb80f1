"""Python binding of libflux_attn.so (the C-ABI in include/flux_attn.h).

Argument marshalling only: torch supplies device memory and streams, every
step of the computation runs in the library's kernels. There is no fallback:
a missing library, a CPU tensor or a non-zero status raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

AXES_DIMS = (32, 32, 32, 32)
THETA = 2000.0

STATUS = {
    0: "FLUX_OK", -1: "FLUX_ERR_NULL", -2: "FLUX_ERR_SHAPE", -3: "FLUX_ERR_AXES",
    -4: "FLUX_ERR_ALIGN", -5: "FLUX_ERR_WORKSPACE", -6: "FLUX_ERR_CUDA",
    -7: "FLUX_ERR_DEVICE_TIMEOUT", -8: "FLUX_ERR_UNSUPPORTED", -9: "FLUX_ERR_ALIAS",
}

# every symbol include/flux_attn.h declares
EXPORTS = ("flux_rope_tables", "flux_rope_tables_packed", "flux_joint_rope_attention_workspace",
           "flux_joint_rope_attention_krot_bytes", "flux_joint_rope_attention_workspace_shared",
           "flux_joint_rope_attention", "flux_joint_rope_attention_tabled",
           "flux_joint_rope_attention_heads", "flux_joint_rope_attention_rows",
           "flux_joint_rope_attention_rows_workspace",
           "flux_joint_qknorm_rope_attention", "flux_joint_qknorm_rope_attention_tabled",
           "flux_joint_rope_attention_extract_workspace", "flux_joint_rope_attention_extract",
           "flux_joint_rope_attention_cached_workspace", "flux_joint_rope_attention_cached",
           "flux_joint_qknorm_rope_attention_extract", "flux_joint_qknorm_rope_attention_cached",
           "flux_qkv_mlp_proj", "flux_linear", "flux_modulated_norm", "flux_quantize_fp8",
           "flux_linear_fp8", "flux_cross_attention", "flux_query_status", "flux_status_word",
           "flux_take_status", "flux_status_string")


class FluxError(RuntimeError):
    def __init__(self, fn: str, status: int, lib=None):
        msg = lib.flux_status_string(status).decode() if lib is not None else ""
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({msg})")
        self.status = status


_lock = threading.Lock()
_lib = None
_compiled = None  # the compiled marshalling, and the library that it calls
_compiled_lib = None


def _load_compiled(lib):
    """The compiled marshalling (build.build_marshal) of the calls that have one, over
    `lib`; without it, or without torch, they are marshalled here. A file that does not
    load is warned of and passed over."""
    global _compiled, _compiled_lib
    import importlib.util

    try:
        path = _build.marshal_path()
    except (ImportError, OSError):  # no torch, or no sources to tell the file by
        return
    if not os.path.exists(path):
        return
    try:
        spec = importlib.util.spec_from_file_location("_marshal", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError as e:
        import warnings

        warnings.warn(f"the compiled marshalling does not load ({e}): calls are marshalled in "
                      "Python", RuntimeWarning)
        return
    module.bind(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in
                  ("flux_quantize_fp8", "flux_linear_fp8", "flux_cross_attention")))
    _compiled, _compiled_lib = module, lib


def library_path() -> str:
    """FLUX_ATTN_LIB if set; else the checked build when FLUX_ATTN_DEBUG=1
    (build it with ``python -m diffusion_transformer_joint_gb300.build
    --checked``); else the release build."""
    if "FLUX_ATTN_LIB" in os.environ:
        return os.environ["FLUX_ATTN_LIB"]
    if os.environ.get("FLUX_ATTN_DEBUG") == "1":
        return _build.CHECKED_LIB_PATH
    return _build.LIB_PATH


def load(path: str | None = None):
    """Load (once) and return the ctypes handle; raises if the library is missing."""
    global _lib
    with _lock:
        if _lib is None:
            p = path or library_path()
            if not os.path.exists(p):
                raise RuntimeError(f"CUDA library not built: {p} (run "
                                   "python -m diffusion_transformer_joint_gb300.build)")
            lib = ctypes.CDLL(p)
            V, I64, I32, SZ, D = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                  ctypes.c_size_t, ctypes.c_double)
            lib.flux_rope_tables.argtypes = [V, I64, V, I32, D, V, V, V]
            lib.flux_rope_tables.restype = I32
            lib.flux_rope_tables_packed.argtypes = [V, I64, V, I32, D, V, V]
            lib.flux_rope_tables_packed.restype = I32
            lib.flux_joint_rope_attention_workspace.argtypes = [I64, I32]
            lib.flux_joint_rope_attention_workspace.restype = SZ
            lib.flux_joint_rope_attention_krot_bytes.argtypes = [I32, I64, I32, I32]
            lib.flux_joint_rope_attention_krot_bytes.restype = SZ
            lib.flux_joint_rope_attention_workspace_shared.argtypes = [I32, I64, I32, I32]
            lib.flux_joint_rope_attention_workspace_shared.restype = SZ
            lib.flux_joint_rope_attention.argtypes = [V, V, V, V, I64, V, I64, I32, I32, I32,
                                                      V, I32, D, V, V, SZ, V]
            lib.flux_joint_rope_attention.restype = I32
            lib.flux_joint_rope_attention_tabled.argtypes = [V, V, V, V, I32, I64, I32, I32, V,
                                                             V, V, SZ, V]
            lib.flux_joint_rope_attention_heads.argtypes = [V, V, V, V, I64, V, I64, I32, I32,
                                                            I32, I32, I32, V, I32, D, V, V, SZ, V]
            lib.flux_joint_rope_attention_heads.restype = I32
            lib.flux_joint_rope_attention_rows.argtypes = [V, I64, I64, V, V, V, I64, V, I64, I32,
                                                           I32, I32, V, I32, D, V, V, SZ, V]
            lib.flux_joint_rope_attention_rows.restype = I32
            lib.flux_joint_rope_attention_rows_workspace.argtypes = [I32, I64, I64, I32, I32]
            lib.flux_joint_rope_attention_rows_workspace.restype = SZ
            lib.flux_joint_rope_attention_tabled.restype = I32
            F = ctypes.c_float
            lib.flux_joint_qknorm_rope_attention.argtypes = [
                V, V, V, V, I64, V, I64, I32, I32, I32, V, I32, D, V, V, V, V, F, V, V, SZ, V]
            lib.flux_joint_qknorm_rope_attention.restype = I32
            lib.flux_joint_qknorm_rope_attention_tabled.argtypes = [
                V, V, V, V, I32, I64, I32, I32, I64, V, V, V, V, F, V, V, V, SZ, V]
            lib.flux_joint_qknorm_rope_attention_tabled.restype = I32
            lib.flux_joint_rope_attention_extract_workspace.argtypes = [I32, I64, I64, I64, I32, I32]
            lib.flux_joint_rope_attention_extract_workspace.restype = SZ
            lib.flux_joint_rope_attention_extract.argtypes = [
                V, V, V, V, I64, V, I64, V, I64, I32, I32, I32, V, I32, D, V, V, V, V, SZ, V]
            lib.flux_joint_rope_attention_extract.restype = I32
            lib.flux_joint_rope_attention_cached_workspace.argtypes = [I32, I64, I64, I64, I32, I32]
            lib.flux_joint_rope_attention_cached_workspace.restype = SZ
            lib.flux_joint_rope_attention_cached.argtypes = [
                V, V, V, V, I64, V, I64, V, V, I64, I32, I32, I32, V, I32, D, V, V, SZ, V]
            lib.flux_joint_rope_attention_cached.restype = I32
            lib.flux_joint_qknorm_rope_attention_extract.argtypes = [
                V, V, V, V, I64, V, I64, V, I64, I32, I32, I32, V, I32, D, V, V, V, V, F, V, V, V, V,
                SZ, V]
            lib.flux_joint_qknorm_rope_attention_extract.restype = I32
            lib.flux_joint_qknorm_rope_attention_cached.argtypes = [
                V, V, V, V, I64, V, I64, V, V, I64, I32, I32, I32, V, I32, D, V, V, V, V, F, V, V,
                SZ, V]
            lib.flux_joint_qknorm_rope_attention_cached.restype = I32
            lib.flux_qkv_mlp_proj.argtypes = [V, V, I64, I32, I32, I32, I64, V, V, V, V, V, V]
            lib.flux_qkv_mlp_proj.restype = I32
            lib.flux_linear.argtypes = [V, I64, I64, I32, V, I64, I64, I32, V, I64, I32, I64, I64,
                                        I32, V, V, I64, I32, V, I64, I64, V, I64, I64, V, V]
            lib.flux_linear.restype = I32
            lib.flux_modulated_norm.argtypes = [V, I64, I64, I32, V, I64, I64, V, I64, V, I64, V,
                                                I64, I32, I32, I64, I32, I32, F, V, I64, I64, V,
                                                I64, I64, V]
            lib.flux_modulated_norm.restype = I32
            lib.flux_quantize_fp8.argtypes = [V, I64, I64, I32, I32, I64, I32, I32, V, I64, I64, V,
                                              I64, I64, I64, V]
            lib.flux_quantize_fp8.restype = I32
            lib.flux_linear_fp8.argtypes = [V, I64, I64, V, I64, I64, I64, V, I64, V, I64, I64,
                                            I32, I64, I32, I64, I32, V, V, I64, I32, V, I64, I64,
                                            V, I64, I64, V, V]
            lib.flux_linear_fp8.restype = I32
            lib.flux_cross_attention.argtypes = [V, I64, I64, V, I64, I64, V, I64, I64, V, V, I64,
                                                 I32, I64, I64, I32, I32, I32, F, V, I64, I64, V, V]
            lib.flux_cross_attention.restype = I32
            lib.flux_query_status.argtypes = [V, V]
            lib.flux_query_status.restype = I32
            lib.flux_status_word.argtypes = [V]
            lib.flux_status_word.restype = I32
            lib.flux_take_status.argtypes = [V]
            lib.flux_take_status.restype = I32
            lib.flux_status_string.argtypes = [I32]
            lib.flux_status_string.restype = ctypes.c_char_p
            _load_compiled(lib)
            _lib = lib
    return _lib


def _axes_array(axes_dims):
    arr = (ctypes.c_int32 * len(axes_dims))(*[int(a) for a in axes_dims])
    return arr, len(axes_dims)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None and t.numel() > 0 else None


def _stream_handle(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need_cuda(name, t, dtype):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_shape(name, t, shape):
    """The C ABI takes pointers and sizes only: every tensor's shape is checked
    here, before a kernel could read or write past it."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _need_ids(name, ids, n_axes):
    if ids is not None and ids.numel() > 0 and (ids.dim() != 2 or int(ids.shape[1]) != n_axes):
        raise ValueError(f"{name} must be [tokens, {n_axes}], got {tuple(ids.shape)}")


def workspace_bytes(S: int, D: int = 128) -> int:
    """Smallest workspace of joint_rope_attention (status word + RoPE table)."""
    return int(load().flux_joint_rope_attention_workspace(int(S), int(D)))


def krot_bytes(B: int, S: int, H: int, D: int = 128) -> int:
    """Size of the rotated-K exchange buffer (0 for rejected shapes)."""
    return int(load().flux_joint_rope_attention_krot_bytes(int(B), int(S), int(H), int(D)))


def workspace_shared_bytes(B: int, S: int, H: int, D: int = 128) -> int:
    """Workspace size with which joint_rope_attention shares rotated K tiles."""
    return int(load().flux_joint_rope_attention_workspace_shared(int(B), int(S), int(H), int(D)))


def extract_workspace_bytes(B: int, S_txt: int, S_ref: int, S_img: int, H: int,
                            D: int = 128) -> int:
    """Workspace size of one attention_extract call (0: bad shape)."""
    return int(load().flux_joint_rope_attention_extract_workspace(int(B), int(S_txt), int(S_ref),
                                                                 int(S_img), int(H), int(D)))


def cached_workspace_bytes(B: int, S_txt: int, S_img: int, S_ref: int, H: int,
                           D: int = 128) -> int:
    """Workspace size of one attention_cached call (0: bad shape)."""
    return int(load().flux_joint_rope_attention_cached_workspace(int(B), int(S_txt), int(S_img),
                                                                int(S_ref), int(H), int(D)))


def rope_tables(ids, axes_dims=AXES_DIMS, theta=THETA, cos_out=None, sin_out=None, stream=None):
    """fp32 cos, sin [S, sum(axes_dims)/2] for int32 ids [S, n_axes] on the GPU."""
    import torch

    lib = load()
    _need_cuda("ids", ids, torch.int32)
    S, n_axes = ids.shape
    P = sum(int(a) for a in axes_dims) // 2
    if cos_out is None:
        cos_out = torch.empty((S, P), dtype=torch.float32, device=ids.device)
    if sin_out is None:
        sin_out = torch.empty((S, P), dtype=torch.float32, device=ids.device)
    for name, t in (("cos_out", cos_out), ("sin_out", sin_out)):
        _need_cuda(name, t, torch.float32)
        _need_shape(name, t, (S, P))
    axes, n = _axes_array(axes_dims)
    if n != n_axes:
        raise ValueError("ids' last dimension must equal len(axes_dims)")
    rc = lib.flux_rope_tables(_ptr(ids), S, axes, n, float(theta), _ptr(cos_out), _ptr(sin_out),
                              _stream_handle(stream))
    if rc != 0:
        raise FluxError("flux_rope_tables", rc, lib)
    return cos_out, sin_out


def rope_tables_packed(ids, axes_dims=AXES_DIMS, theta=THETA, out=None, stream=None):
    """Packed table [S, sum(axes_dims)/2] (int32 storage of uint32 words: fp16 cos
    in bits 0-15, fp16 sin in bits 16-31) for int32 ids [S, n_axes] on the GPU."""
    import torch

    lib = load()
    _need_cuda("ids", ids, torch.int32)
    S, n_axes = ids.shape
    P = sum(int(a) for a in axes_dims) // 2
    if out is None:
        out = torch.empty((S, P), dtype=torch.int32, device=ids.device)
    _need_cuda("out", out, torch.int32)
    _need_shape("out", out, (S, P))
    axes, n = _axes_array(axes_dims)
    if n != n_axes:
        raise ValueError("ids' last dimension must equal len(axes_dims)")
    rc = lib.flux_rope_tables_packed(_ptr(ids), S, axes, n, float(theta), _ptr(out),
                                     _stream_handle(stream))
    if rc != 0:
        raise FluxError("flux_rope_tables_packed", rc, lib)
    return out


def unpack_table(packed):
    """(cos, sin) fp32 tensors from a packed table (the fp16 halves, widened)."""
    import torch

    w = packed.contiguous()
    halves = w.view(torch.int16).view(torch.float16).reshape(*w.shape, 2)
    return halves[..., 0].float(), halves[..., 1].float()


def _norm_args(qk_norm, device, D=128):
    """(q_txt, k_txt, q_img, k_img, eps) -> four fp32 CUDA [D] tensors and eps
    (the kernels read D weights from each pointer)."""
    import torch

    if len(qk_norm) != 5:
        raise ValueError("qk_norm must be (q_norm_txt, k_norm_txt, q_norm_img, k_norm_img, eps)")
    *ws, eps = qk_norm
    names = ("q_norm_txt", "k_norm_txt", "q_norm_img", "k_norm_img")
    ts = [w if isinstance(w, torch.Tensor) else torch.as_tensor(w, dtype=torch.float32,
                                                                device=device) for w in ws]
    for name, w in zip(names, ts):
        _need_shape(name, w, (D,))
    for name, w in zip(names, ts):
        _need_cuda(name, w, torch.float32)
    return ts, float(eps)


def joint_rope_attention(q, k, v, txt_ids, img_ids, axes_dims=AXES_DIMS, theta=THETA, out=None,
                         workspace=None, stream=None, share_k=True, qk_norm=None):
    """softmax(RoPE(q) RoPE(k)^T / sqrt(D)) v over the joint sequence [txt ; img].

    q, k, v: bf16 CUDA [B, S, H, 128]; txt_ids [S_txt, n_axes], img_ids
    [S_img, n_axes] int32 CUDA (either may be None / empty). Returns ``out``.
    Without ``workspace`` one is allocated: with room for the rotated-K
    exchange buffer when ``share_k``, else the smallest one. ``qk_norm``:
    None, or (q_norm_txt, k_norm_txt, q_norm_img, k_norm_img, eps) with fp32
    [128] weights, for the QK RMS normalisation before RoPE.
    """
    import torch

    lib = load()
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need_cuda(name, t, torch.bfloat16)
    B, S, H, D = q.shape
    _need_shape("k", k, q.shape)
    _need_shape("v", v, q.shape)
    S_txt = 0 if txt_ids is None else int(txt_ids.shape[0])
    S_img = 0 if img_ids is None else int(img_ids.shape[0])
    for name, t in (("txt_ids", txt_ids), ("img_ids", img_ids)):
        if t is not None and t.numel() > 0:
            _need_cuda(name, t, torch.int32)
            _need_ids(name, t, len(axes_dims))
    if S_txt + S_img != S:
        raise ValueError(f"the ids give {S_txt} + {S_img} tokens, q has {S}")
    if out is None:
        out = torch.empty_like(q)
    else:
        _need_cuda("out", out, torch.bfloat16)
        _need_shape("out", out, q.shape)
    if workspace is not None:
        _need_cuda("workspace", workspace, torch.uint8)
    if workspace is None:
        n = workspace_shared_bytes(B, S, H, D) if share_k else 0
        if n == 0:
            n = workspace_bytes(max(S, 1), D)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    axes, n = _axes_array(axes_dims)
    if qk_norm is None:
        rc = lib.flux_joint_rope_attention(
            _ptr(q), _ptr(k), _ptr(v), _ptr(txt_ids), S_txt, _ptr(img_ids), S_img, B, H, D, axes,
            n, float(theta), _ptr(out), _ptr(workspace), workspace.numel(), _stream_handle(stream))
        name = "flux_joint_rope_attention"
    else:
        ws, eps = _norm_args(qk_norm, q.device, D)
        rc = lib.flux_joint_qknorm_rope_attention(
            _ptr(q), _ptr(k), _ptr(v), _ptr(txt_ids), S_txt, _ptr(img_ids), S_img, B, H, D, axes,
            n, float(theta), *[_ptr(w) for w in ws], eps, _ptr(out), _ptr(workspace),
            workspace.numel(), _stream_handle(stream))
        name = "flux_joint_qknorm_rope_attention"
    if rc != 0:
        raise FluxError(name, rc, lib)
    return out


def _check_ids(txt_ids, img_ids, n_axes):
    import torch

    for name, t in (("txt_ids", txt_ids), ("img_ids", img_ids)):
        if t is not None and t.numel() > 0:
            _need_cuda(name, t, torch.int32)
            _need_ids(name, t, n_axes)
    return (0 if txt_ids is None else int(txt_ids.shape[0]),
            0 if img_ids is None else int(img_ids.shape[0]))


def joint_rope_attention_heads(q, k, v, txt_ids, img_ids, h0, n_heads, axes_dims=AXES_DIMS,
                               theta=THETA, out=None, workspace=None, stream=None, share_k=True):
    """joint_rope_attention over heads h0 .. h0 + n_heads - 1 of the [B, S, H, 128]
    tensors q, k, v (a tensor-parallel rank's heads); only those heads of
    ``out`` are written (it is allocated, and left uninitialised elsewhere,
    when None)."""
    import torch

    lib = load()
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need_cuda(name, t, torch.bfloat16)
    B, S, H, D = q.shape
    _need_shape("k", k, q.shape)
    _need_shape("v", v, q.shape)
    S_txt, S_img = _check_ids(txt_ids, img_ids, len(axes_dims))
    if S_txt + S_img != S:
        raise ValueError(f"the ids give {S_txt} + {S_img} tokens, q has {S}")
    if out is None:
        out = torch.empty_like(q)
    else:
        _need_cuda("out", out, torch.bfloat16)
        _need_shape("out", out, q.shape)
    if workspace is None:
        n = workspace_shared_bytes(B, S, int(n_heads), D) if share_k else 0
        workspace = torch.empty(max(n or workspace_bytes(S, D), 256), dtype=torch.uint8,
                                device=q.device)
    else:
        _need_cuda("workspace", workspace, torch.uint8)
    axes, n = _axes_array(axes_dims)
    rc = lib.flux_joint_rope_attention_heads(
        _ptr(q), _ptr(k), _ptr(v), _ptr(txt_ids), S_txt, _ptr(img_ids), S_img, B, H, int(h0),
        int(n_heads), D, axes, n, float(theta), _ptr(out), _ptr(workspace), workspace.numel(),
        _stream_handle(stream))
    if rc != 0:
        raise FluxError("flux_joint_rope_attention_heads", rc, lib)
    return out


def rows_workspace_bytes(B: int, S_q: int, S: int, H: int, D: int = 128) -> int:
    """Workspace of joint_rope_attention_rows with the exchange buffer."""
    return int(load().flux_joint_rope_attention_rows_workspace(int(B), int(S_q), int(S), int(H),
                                                               int(D)))


def joint_rope_attention_rows(q, q0, k, v, txt_ids, img_ids, axes_dims=AXES_DIMS, theta=THETA,
                              out=None, workspace=None, stream=None, share_k=True):
    """The attention of query tokens q0 .. q0 + S_q - 1 (q: bf16 [B, S_q, H, 128])
    over every token's key and value (k, v: [B, S, H, 128]); txt_ids / img_ids
    are the ids of the whole sequence. Returns out [B, S_q, H, 128]."""
    import torch

    lib = load()
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need_cuda(name, t, torch.bfloat16)
    B, S_q, H, D = q.shape
    S = k.shape[1]
    _need_shape("k", k, (B, S, H, D))
    _need_shape("v", v, (B, S, H, D))
    S_txt, S_img = _check_ids(txt_ids, img_ids, len(axes_dims))
    if S_txt + S_img != S:
        raise ValueError(f"the ids give {S_txt} + {S_img} tokens, k has {S}")
    if out is None:
        out = torch.empty_like(q)
    else:
        _need_cuda("out", out, torch.bfloat16)
        _need_shape("out", out, q.shape)
    if workspace is None:
        n = rows_workspace_bytes(B, S_q, S, H, D) if share_k else 0
        workspace = torch.empty(max(n or workspace_bytes(S, D), 256), dtype=torch.uint8,
                                device=q.device)
    else:
        _need_cuda("workspace", workspace, torch.uint8)
    axes, n = _axes_array(axes_dims)
    rc = lib.flux_joint_rope_attention_rows(
        _ptr(q), int(q0), S_q, _ptr(k), _ptr(v), _ptr(txt_ids), S_txt, _ptr(img_ids), S_img, B,
        H, D, axes, n, float(theta), _ptr(out), _ptr(workspace), workspace.numel(),
        _stream_handle(stream))
    if rc != 0:
        raise FluxError("flux_joint_rope_attention_rows", rc, lib)
    return out


def joint_rope_attention_tabled(q, k, v, table, status, out=None, stream=None, krot=None,
                                qk_norm=None, s_txt=0):
    """Attention with a caller-built packed table (see rope_tables_packed); ``status``
    is a device int32 tensor of one element that the caller clears. ``krot``: a
    uint8 CUDA tensor of at least krot_bytes(B, S, H) bytes serving as the
    rotated-K exchange buffer; None allocates one, False runs without.
    ``qk_norm`` as for joint_rope_attention, with ``s_txt`` leading text tokens."""
    import torch

    lib = load()
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need_cuda(name, t, torch.bfloat16)
    _need_cuda("table", table, torch.int32)
    _need_cuda("status", status, torch.int32)
    B, S, H, D = q.shape
    _need_shape("k", k, q.shape)
    _need_shape("v", v, q.shape)
    _need_shape("table", table, (S, D // 2))
    if status.numel() < 1:
        raise ValueError("status must hold one int32")
    if out is None:
        out = torch.empty_like(q)
    else:
        _need_cuda("out", out, torch.bfloat16)
        _need_shape("out", out, q.shape)
    if krot is None:
        krot = torch.empty(max(krot_bytes(B, S, H, D), 256), dtype=torch.uint8, device=q.device)
    if krot is False:
        kp, kn = None, 0
    else:
        _need_cuda("krot", krot, torch.uint8)
        kp, kn = _ptr(krot), krot.numel()
    if qk_norm is None:
        rc = lib.flux_joint_rope_attention_tabled(_ptr(q), _ptr(k), _ptr(v), _ptr(table), B, S, H,
                                                  D, _ptr(out), _ptr(status), kp, kn,
                                                  _stream_handle(stream))
        name = "flux_joint_rope_attention_tabled"
    else:
        ws, eps = _norm_args(qk_norm, q.device, D)
        rc = lib.flux_joint_qknorm_rope_attention_tabled(
            _ptr(q), _ptr(k), _ptr(v), _ptr(table), B, S, H, D, int(s_txt),
            *[_ptr(w) for w in ws], eps, _ptr(out), _ptr(status), kp, kn, _stream_handle(stream))
        name = "flux_joint_qknorm_rope_attention_tabled"
    if rc != 0:
        raise FluxError(name, rc, lib)
    return out


def _rows(ids):
    return 0 if ids is None else int(ids.shape[0])


def attention_extract(q, k, v, txt_ids, ref_ids, img_ids, axes_dims=AXES_DIMS, theta=THETA,
                      out=None, cache_k=None, cache_v=None, workspace=None, stream=None,
                      qk_norm=None):
    """Extract mode over tokens [txt ; ref ; img]: returns (out, cache_k, cache_v).
    ``qk_norm`` as for joint_rope_attention (reference tokens take the image
    weights; the cache then holds the normalised, rotated K)."""
    import torch

    lib = load()
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need_cuda(name, t, torch.bfloat16)
    B, S, H, D = q.shape
    _need_shape("k", k, q.shape)
    _need_shape("v", v, q.shape)
    s_t, s_r, s_i = _rows(txt_ids), _rows(ref_ids), _rows(img_ids)
    for name, t in (("txt_ids", txt_ids), ("ref_ids", ref_ids), ("img_ids", img_ids)):
        if t is not None and t.numel() > 0:
            _need_cuda(name, t, torch.int32)
            _need_ids(name, t, len(axes_dims))
    if s_t + s_r + s_i != S:
        raise ValueError(f"the ids give {s_t} + {s_r} + {s_i} tokens, q has {S}")
    out = torch.empty_like(q) if out is None else out
    if cache_k is None:
        cache_k = torch.empty((B, s_r, H, D), dtype=torch.bfloat16, device=q.device)
    if cache_v is None:
        cache_v = torch.empty((B, s_r, H, D), dtype=torch.bfloat16, device=q.device)
    for name, t, shape in (("out", out, q.shape), ("cache_k", cache_k, (B, s_r, H, D)),
                           ("cache_v", cache_v, (B, s_r, H, D))):
        _need_cuda(name, t, torch.bfloat16)
        _need_shape(name, t, shape)
    if workspace is not None:
        _need_cuda("workspace", workspace, torch.uint8)
    if workspace is None:
        n = extract_workspace_bytes(B, s_t, s_r, s_i, H, D)
        workspace = torch.empty(max(int(n), 256), dtype=torch.uint8, device=q.device)
    axes, na = _axes_array(axes_dims)
    if qk_norm is None:
        name = "flux_joint_rope_attention_extract"
        rc = lib.flux_joint_rope_attention_extract(
            _ptr(q), _ptr(k), _ptr(v), _ptr(txt_ids), s_t, _ptr(ref_ids), s_r, _ptr(img_ids), s_i,
            B, H, D, axes, na, float(theta), _ptr(out), _ptr(cache_k), _ptr(cache_v),
            _ptr(workspace), workspace.numel(), _stream_handle(stream))
    else:
        name = "flux_joint_qknorm_rope_attention_extract"
        ws, eps = _norm_args(qk_norm, q.device, D)
        rc = lib.flux_joint_qknorm_rope_attention_extract(
            _ptr(q), _ptr(k), _ptr(v), _ptr(txt_ids), s_t, _ptr(ref_ids), s_r, _ptr(img_ids), s_i,
            B, H, D, axes, na, float(theta), *[_ptr(w) for w in ws], eps, _ptr(out),
            _ptr(cache_k), _ptr(cache_v), _ptr(workspace), workspace.numel(),
            _stream_handle(stream))
    if rc != 0:
        raise FluxError(name, rc, lib)
    return out, cache_k, cache_v


def attention_cached(q, k, v, txt_ids, img_ids, cache_k, cache_v, axes_dims=AXES_DIMS,
                     theta=THETA, out=None, workspace=None, stream=None, qk_norm=None):
    """Cached mode: queries [txt ; img] over keys [txt ; cache ; img]; returns out.
    ``qk_norm`` normalises q and the keys of k (the cache is used as stored)."""
    import torch

    lib = load()
    for name, t in (("q", q), ("k", k), ("v", v), ("cache_k", cache_k), ("cache_v", cache_v)):
        _need_cuda(name, t, torch.bfloat16)
    B, S, H, D = q.shape
    _need_shape("k", k, q.shape)
    _need_shape("v", v, q.shape)
    s_t, s_i, s_r = _rows(txt_ids), _rows(img_ids), int(cache_k.shape[1])
    _need_shape("cache_k", cache_k, (B, s_r, H, D))
    _need_shape("cache_v", cache_v, (B, s_r, H, D))
    for name, t in (("txt_ids", txt_ids), ("img_ids", img_ids)):
        if t is not None and t.numel() > 0:
            _need_cuda(name, t, torch.int32)
            _need_ids(name, t, len(axes_dims))
    if s_t + s_i != S:
        raise ValueError(f"the ids give {s_t} + {s_i} tokens, q has {S}")
    out = torch.empty_like(q) if out is None else out
    _need_cuda("out", out, torch.bfloat16)
    _need_shape("out", out, q.shape)
    if workspace is not None:
        _need_cuda("workspace", workspace, torch.uint8)
    if workspace is None:
        n = cached_workspace_bytes(B, s_t, s_i, s_r, H, D)
        workspace = torch.empty(max(int(n), 256), dtype=torch.uint8, device=q.device)
    axes, na = _axes_array(axes_dims)
    if qk_norm is None:
        name = "flux_joint_rope_attention_cached"
        rc = lib.flux_joint_rope_attention_cached(
            _ptr(q), _ptr(k), _ptr(v), _ptr(txt_ids), s_t, _ptr(img_ids), s_i, _ptr(cache_k),
            _ptr(cache_v), s_r, B, H, D, axes, na, float(theta), _ptr(out), _ptr(workspace),
            workspace.numel(), _stream_handle(stream))
    else:
        name = "flux_joint_qknorm_rope_attention_cached"
        ws, eps = _norm_args(qk_norm, q.device, D)
        rc = lib.flux_joint_qknorm_rope_attention_cached(
            _ptr(q), _ptr(k), _ptr(v), _ptr(txt_ids), s_t, _ptr(img_ids), s_i, _ptr(cache_k),
            _ptr(cache_v), s_r, B, H, D, axes, na, float(theta), *[_ptr(w) for w in ws], eps,
            _ptr(out), _ptr(workspace), workspace.numel(), _stream_handle(stream))
    if rc != 0:
        raise FluxError(name, rc, lib)
    return out


def qkv_mlp_proj(x, w, H, mlp=None, q=None, k=None, v=None, act=None, status=None,
                 stream=None):
    """Fused single-stream input projection: x [..., dim] and w [3 H 128 + 2 mlp, dim]
    bf16 -> (q, k, v [..., H, 128], act [..., mlp]); status (int32 [1]) receives a
    device timeout, without it the device's own word (take_status)."""
    import torch

    lib = load()
    _need_cuda("x", x, torch.bfloat16)
    _need_cuda("w", w, torch.bfloat16)
    lead, dim = tuple(x.shape[:-1]), int(x.shape[-1])
    M = 1
    for n in lead:
        M *= int(n)
    inner = H * 128
    if mlp is None:
        mlp = (int(w.shape[0]) - 3 * inner) // 2
    if mlp < 0:
        raise ValueError(f"w has {int(w.shape[0])} rows, fewer than the {3 * inner} of q, k, v")
    if tuple(w.shape) != (3 * inner + 2 * mlp, dim):
        raise ValueError(f"w must be [{3 * inner + 2 * mlp}, {dim}], got {tuple(w.shape)}")
    dev = x.device
    q = torch.empty(lead + (H, 128), dtype=torch.bfloat16, device=dev) if q is None else q
    k = torch.empty(lead + (H, 128), dtype=torch.bfloat16, device=dev) if k is None else k
    v = torch.empty(lead + (H, 128), dtype=torch.bfloat16, device=dev) if v is None else v
    if act is None:
        act = torch.empty(lead + (mlp,), dtype=torch.bfloat16, device=dev)
    for name, t in (("q", q), ("k", k), ("v", v), ("act", act)):
        _need_cuda(name, t, torch.bfloat16)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need_shape(name, t, lead + (H, 128))
    _need_shape("act", act, lead + (mlp,))
    if status is None:
        sp = _own_status(lib, torch.cuda.current_device())
    else:
        _need_cuda("status", status, torch.int32)
        sp = _ptr(status)
    rc = lib.flux_qkv_mlp_proj(_ptr(x), _ptr(w), M, dim, int(H), 128, int(mlp), _ptr(q), _ptr(k),
                               _ptr(v), _ptr(act) if mlp > 0 else None, sp,
                               _stream_handle(stream))
    if rc != 0:
        raise FluxError("flux_qkv_mlp_proj", rc, lib)
    return q, k, v, act


ACTIVATIONS = {None: 0, "silu": 1, "gelu_tanh": 2, "swiglu": 3}
NORMS = {"layer": 0, "rms": 1}


def _token_rows(name, t, shape, dtype, dev):
    """(address, batch stride, token stride) of a tensor of token rows on CUDA
    device `dev`, [B, S, width] or [S, width] with contiguous channels; raises
    for anything else."""
    st = t.stride()
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev or st[-1] != 1:
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.get_device() != dev:
            raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
        raise ValueError(f"{name} must have contiguous channels, got strides {st}")
    return (t.data_ptr(), *st[:2]) if len(st) == 3 else (t.data_ptr(), 0, st[0])


def _vector(name, t, B, width, dtype, dev):
    """(address, batch stride) of a vector [width], or of one per batch element
    [B, width] (a stride of 0 where all are the same)."""
    shape, st = t.shape, t.stride()
    n = len(shape)
    if n == 2:
        bs = st[0] if shape[0] == B and B > 1 else 0
        if shape[0] not in (1, B) or shape[1] != width:
            n = 0
    elif n != 1 or shape[0] != width:
        n = 0
    if n == 0:
        raise ValueError(f"{name} must be [{width}] or [{B}, {width}], got {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} like the other vectors, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    if st[-1] != 1 and width > 1:
        raise ValueError(f"{name} must be contiguous, got strides {st}")
    return t.data_ptr(), bs if n == 2 else 0


def _vector_type(dtype):
    """vec_f32 of a call whose vectors have this type."""
    import torch

    if dtype == torch.bfloat16:
        return 0
    if dtype != torch.float32:
        raise ValueError(f"bias, gate, scale and shift must be bfloat16 or float32, got {dtype}")
    return 1


def _stream_of(x, stream):
    """(device index, stream handle) of a call on x's device, which must be current."""
    import torch

    dev = torch.cuda.current_device() if x.is_cuda else None
    if dev is None:
        raise ValueError("x must be a CUDA tensor (no CPU path exists)")
    if x.get_device() != dev:
        raise ValueError(f"x is on {x.device}, the current device is cuda:{dev}")
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"the stream is on {stream.device}, x on {x.device}")
    return dev, stream.cuda_stream


def _allocate(stream, fn, *args, **kw):
    """Memory of the stream that uses it: fn(*args) under `stream` (None: the
    current one)."""
    import torch

    if stream is None:
        return fn(*args, **kw)
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def linear(x, w, x2=None, bias=None, act=None, gate=None, residual=None, out=None, status=None,
           stream=None):
    """A linear layer with its epilogue: residual + gate * act([x | x2] W^T + bias).

    x: bf16 CUDA [B, S, K] (or [S, K]); x2 more input channels [B, S, K2]; w
    bf16 [N, K + K2], or [2 N, K + K2] for act "swiglu" (the gate rows, then the
    linear rows). act: None, "silu", "gelu_tanh" or "swiglu". bias [N] ([2 N])
    and gate [N] or [B, N] are both bf16 or both fp32; residual and ``out`` are
    bf16 [B, S, N] (``out=residual`` updates a stream in place). Token tensors
    and w may have strides between rows and batch elements (views of a joint
    sequence, of a wider buffer or of w's columns). ``status`` (int32 [1])
    receives a device timeout, without it the device's own word (take_status).
    Returns out.
    """
    import torch

    lib = _lib or load()
    dev, handle = _stream_of(x, stream)
    bf16, shape = torch.bfloat16, x.shape
    if len(shape) not in (2, 3):
        raise ValueError(f"x must be [B, S, K] or [S, K], got {tuple(shape)}")
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {list(ACTIVATIONS)}, got {act!r}")
    B, S, K = shape if len(shape) == 3 else (1, *shape)
    K2 = 0 if x2 is None else x2.shape[-1]
    if B > 0x7FFFFFFF or K > 0x7FFFFFFF or K2 > 0x7FFFFFFF:
        raise ValueError(f"batch and channels must be below 2^31, got {B}, {K}, {K2}")
    xp, xb, xr = _token_rows("x", x, shape, bf16, dev)
    if w.dim() != 2 or w.shape[1] != K + K2:
        raise ValueError(f"w must be [rows, {K + K2}], got {tuple(w.shape)}")
    wp, _, wr = _token_rows("w", w, w.shape, bf16, dev)
    rows = N = w.shape[0]
    if act == "swiglu":
        if rows % 2:
            raise ValueError(f"w must have two equal halves of rows, got {rows}")
        N = rows // 2
    shape = (*shape[:-1], N)
    x2p = bp = gp = rp = None
    x2b = x2r = gb = vec_f32 = rb = rr = 0
    if x2 is not None:
        x2p, x2b, x2r = _token_rows("x2", x2, (*shape[:-1], K2), bf16, dev)
    if residual is not None:
        rp, rb, rr = _token_rows("residual", residual, shape, bf16, dev)
    if bias is not None or gate is not None:
        vt = (bias if bias is not None else gate).dtype
        vec_f32 = _vector_type(vt)
        if bias is not None:
            bp = _vector("bias", bias, 1, rows, vt, dev)[0]
        if gate is not None:
            gp, gb = _vector("gate", gate, B, N, vt, dev)
    if out is None:
        out = _allocate(stream, torch.empty, shape, dtype=bf16, device=x.device)
    op, ob, orow = _token_rows("out", out, shape, bf16, dev)
    if status is None:
        sp = _own_words.get(dev) or _own_status(lib, dev)
    elif status.dtype != torch.int32 or status.numel() < 1 or status.get_device() != dev:
        raise ValueError(f"status must hold one int32 on cuda:{dev}")
    else:
        sp = status.data_ptr()
    rc = lib.flux_linear(xp, xb, xr, K, x2p, x2b, x2r, K2, wp, wr, B, S, N, code, bp, gp, gb,
                         vec_f32, rp, rb, rr, op, ob, orow, sp, handle)
    if rc != 0:
        raise FluxError("flux_linear", rc, lib)
    return out


def modulated_norm(x, scale=None, shift=None, y=None, gate=None, norm="layer", eps=1e-6, out=None,
                   x_out=None, stream=None):
    """The modulated norm with the gated residual in front:
    x_out = x + gate * y, h = norm(x_out) * (1 + scale) + shift.

    x: bf16 or fp32 CUDA [B, S, dim] (or [S, dim]); y bf16 of the same shape.
    gate, scale and shift [dim] or [B, dim], all bf16 or all fp32. norm:
    "layer" or "rms", without learned weights. Token tensors may have strides
    between rows and batch elements; ``x_out=x`` updates the stream in place.
    Returns h (bf16, into ``out``), or (h, x_out) when y is given.
    """
    import torch

    lib = _lib or load()
    dev, handle = _stream_of(x, stream)
    bf16, shape, dtype = torch.bfloat16, x.shape, x.dtype
    if len(shape) not in (2, 3):
        raise ValueError(f"x must be [B, S, dim] or [S, dim], got {tuple(shape)}")
    if dtype != bf16 and dtype != torch.float32:
        raise ValueError(f"x must be bfloat16 or float32, got {dtype}")
    kind = NORMS.get(norm)
    if kind is None:
        raise ValueError(f"norm must be one of {list(NORMS)}, got {norm!r}")
    B, S, dim = shape if len(shape) == 3 else (1, *shape)
    if B > 0x7FFFFFFF or dim > 0x7FFFFFFF:
        raise ValueError(f"batch and channels must be below 2^31, got {B}, {dim}")
    xp, xb, xr = _token_rows("x", x, shape, dtype, dev)
    sp = fp = gp = yp = op = None
    sb = fb = gb = yb = yr = ob = orow = vec_f32 = 0
    if scale is not None or shift is not None or gate is not None:
        vt = (scale if scale is not None else shift if shift is not None else gate).dtype
        vec_f32 = _vector_type(vt)
        if scale is not None:
            sp, sb = _vector("scale", scale, B, dim, vt, dev)
        if shift is not None:
            fp, fb = _vector("shift", shift, B, dim, vt, dev)
        if gate is not None:
            gp, gb = _vector("gate", gate, B, dim, vt, dev)
    if out is None:
        out = _allocate(stream, torch.empty, shape, dtype=bf16, device=x.device)
    hp, hb, hr = _token_rows("out", out, shape, bf16, dev)
    if y is not None:
        yp, yb, yr = _token_rows("y", y, shape, bf16, dev)
        if x_out is None:
            x_out = _allocate(stream, torch.empty, shape, dtype=dtype, device=x.device)
        op, ob, orow = _token_rows("x_out", x_out, shape, dtype, dev)
    elif gate is not None or x_out is not None:
        raise ValueError("gate and x_out need y")
    rc = lib.flux_modulated_norm(xp, xb, xr, int(dtype != bf16), yp, yb, yr, gp, gb, sp, sb, fp,
                                 fb, vec_f32, B, S, dim, kind, float(eps), op, ob, orow, hp, hb,
                                 hr, handle)
    if rc != 0:
        raise FluxError("flux_modulated_norm", rc, lib)
    return out if y is None else (out, x_out)


def _done(fn, done, lib):
    """What the compiled marshalling returned: outputs, or the library's status."""
    if type(done) is int:
        raise FluxError(fn, done, lib)
    return done


def _scales(name, t, shape, dev):
    """(address, strides of a group's scales [..., rows, groups]); any strides."""
    import torch

    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != torch.float32:
        raise ValueError(f"{name} must be float32, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    st = t.stride()
    return (t.data_ptr(), *st) if len(st) == 3 else (t.data_ptr(), 0, *st)


def quantize_fp8(x, rows=1, out=None, scale=None, stream=None):
    """Rows or a weight in e4m3 with an fp32 scale per group: scale = t / 448 and
    q = e4m3(x * (448 / t)), t the group's largest magnitude.

    x: bf16 or fp32 CUDA [B, S, K] (or [S, K]), K a multiple of 16, with strides
    between rows and batch elements as for linear. rows: 1, a group is 128
    channels of a row (activations), or 128, it is 128 x 128 of x [N, K]
    (weights). ``out`` is torch.float8_e4m3fn of x's shape; ``scale`` [B, S,
    ceil(K / 128)] ([S, ..]; [ceil(N / 128), ..]) of any strides, made with the
    tokens beside one another. Returns (out, scale).
    """
    import torch

    lib = _lib or load()
    if stream is None and lib is _compiled_lib:
        done = _compiled.quantize_fp8(x, rows, out, scale)
        if done is not None:
            return _done("flux_quantize_fp8", done, lib)
    dev, handle = _stream_of(x, stream)
    e4m3, shape, dtype = torch.float8_e4m3fn, x.shape, x.dtype
    if len(shape) not in (2, 3):
        raise ValueError(f"x must be [B, S, K] or [S, K], got {tuple(shape)}")
    if dtype != torch.bfloat16 and dtype != torch.float32:
        raise ValueError(f"x must be bfloat16 or float32, got {dtype}")
    if rows not in (1, 128) or (rows == 128 and len(shape) != 2):
        raise ValueError(f"rows must be 1, or 128 for x [N, K]; got {rows}, {tuple(shape)}")
    B, S, K = shape if len(shape) == 3 else (1, *shape)
    if B > 0x7FFFFFFF or K > 0x7FFFFFFF:
        raise ValueError(f"batch and channels must be below 2^31, got {B}, {K}")
    xp, xb, xr = _token_rows("x", x, shape, dtype, dev)
    groups = (K + 127) // 128
    if out is None:
        out = _allocate(stream, torch.empty, shape, dtype=e4m3, device=x.device)
    qp, qb, qr = _token_rows("out", out, shape, e4m3, dev)
    lead = shape[:-1] if rows == 1 else ((S + 127) // 128,)
    if scale is None:
        if rows == 1:
            scale = _allocate(stream, torch.empty_strided, (*lead, groups),
                              ((S, 1, B * S) if len(shape) == 3 else (1, S)),
                              dtype=torch.float32, device=x.device)
        else:
            scale = _allocate(stream, torch.empty, (*lead, groups), dtype=torch.float32,
                              device=x.device)
    sp, sb, sr, sk = _scales("scale", scale, (*lead, groups), dev)
    rc = lib.flux_quantize_fp8(xp, xb, xr, int(dtype == torch.float32), B, S, K, rows, qp, qb, qr,
                               sp, sb, sr, sk, handle)
    if rc != 0:
        raise FluxError("flux_quantize_fp8", rc, lib)
    return out, scale


def linear_fp8(x, x_scale, w, w_scale, bias=None, act=None, gate=None, residual=None, out=None,
               status=None, stream=None):
    """A linear layer in 8 bits: residual + gate * act(x W^T + bias), x and W e4m3
    values times their groups' scales (quantize_fp8).

    x: torch.float8_e4m3fn CUDA [B, S, K] (or [S, K]), x_scale fp32 [B, S,
    ceil(K / 128)]; w [N, K] ([2 N, K] for act "swiglu", N a multiple of 128) with
    w_scale [ceil(rows / 128), ceil(K / 128)]. Scales may have any strides. Other
    arguments and the result as for linear.
    """
    import torch

    lib = _lib or load()
    if stream is None and lib is _compiled_lib:
        done = _compiled.linear_fp8(x, x_scale, w, w_scale, bias, act, gate, residual, out, status)
        if done is not None:
            return _done("flux_linear_fp8", done, lib)
    dev, handle = _stream_of(x, stream)
    bf16, e4m3, shape = torch.bfloat16, torch.float8_e4m3fn, x.shape
    if len(shape) not in (2, 3):
        raise ValueError(f"x must be [B, S, K] or [S, K], got {tuple(shape)}")
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {list(ACTIVATIONS)}, got {act!r}")
    B, S, K = shape if len(shape) == 3 else (1, *shape)
    if B > 0x7FFFFFFF or K > 0x7FFFFFFF:
        raise ValueError(f"batch and channels must be below 2^31, got {B}, {K}")
    groups = (K + 127) // 128
    xp, xb, xr = _token_rows("x", x, shape, e4m3, dev)
    xsp, xsb, xsr, xsk = _scales("x_scale", x_scale, (*shape[:-1], groups), dev)
    if w.dim() != 2 or w.shape[1] != K:
        raise ValueError(f"w must be [rows, {K}], got {tuple(w.shape)}")
    wp, _, wr = _token_rows("w", w, w.shape, e4m3, dev)
    rows = N = w.shape[0]
    wsp, _, wsr, wsk = _scales("w_scale", w_scale, ((rows + 127) // 128, groups), dev)
    if act == "swiglu":
        if rows % 2:
            raise ValueError(f"w must have two equal halves of rows, got {rows}")
        N = rows // 2
    shape = (*shape[:-1], N)
    bp = gp = rp = None
    gb = vec_f32 = rb = rr = 0
    if residual is not None:
        rp, rb, rr = _token_rows("residual", residual, shape, bf16, dev)
    if bias is not None or gate is not None:
        vt = (bias if bias is not None else gate).dtype
        vec_f32 = _vector_type(vt)
        if bias is not None:
            bp = _vector("bias", bias, 1, rows, vt, dev)[0]
        if gate is not None:
            gp, gb = _vector("gate", gate, B, N, vt, dev)
    if out is None:
        out = _allocate(stream, torch.empty, shape, dtype=bf16, device=x.device)
    op, ob, orow = _token_rows("out", out, shape, bf16, dev)
    rc = lib.flux_linear_fp8(xp, xb, xr, xsp, xsb, xsr, xsk, wp, wr, wsp, wsr, wsk, B, S, K, N,
                             code, bp, gp, gb, vec_f32, rp, rb, rr, op, ob, orow,
                             _status_pointer(lib, status, dev), handle)
    if rc != 0:
        raise FluxError("flux_linear_fp8", rc, lib)
    return out


def _head_rows(name, t, shape, dev):
    """(address, batch stride, token stride) of bf16 heads [B, S, H, D], a token's
    heads adjacent; raises for anything else."""
    import torch

    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    bs, rs, hs, cs = t.stride()
    if cs != 1 or (hs != shape[3] and shape[2] > 1):
        raise ValueError(f"{name} must have a token's heads adjacent, got strides {t.stride()}")
    return t.data_ptr(), bs, rs


def _softmax_scale(scale):
    """The scale as the library takes it: 0 for its default. What fp32 rounds to 0, which
    would stand for that, is refused, as is what times log2(e) is no longer finite."""
    if scale is None:
        return 0.0
    value = ctypes.c_float(float(scale)).value
    if not 0.0 < value <= 2.0 ** 127:
        raise ValueError(f"scale must be positive in fp32 and at most 2^127, got {scale}")
    return value


def cross_attention(q, k, v, lengths=None, mask=None, scale=None, out=None, status=None,
                    stream=None):
    """Attention to another sequence: softmax(scale q k^T) v over the keys that take part.

    q: bf16 CUDA [B, Sq, H, D], D 64 or 128; k, v bf16 [B, Sk, Hk, D], Hk a
    divisor of H (query heads in groups of H / Hk share a key head); strides
    between tokens and batch elements (two halves of one product's output).
    lengths: int32 [B], keys from there on take no part; mask: bool or uint8 [B,
    Sk], nor do keys where it is 0 (their k and v may hold anything). A row that
    no key is left for is zero. scale: 1 / sqrt(D) unless given; above 0 in fp32, at
    most 2^127. ``out`` bf16 of q's shape; ``status`` as for linear. Returns out.
    """
    import torch

    lib = _lib or load()
    if stream is None and lib is _compiled_lib:
        done = _compiled.cross_attention(q, k, v, lengths, mask, scale, out, status)
        if done is not None:
            return _done("flux_cross_attention", done, lib)
    dev, handle = _stream_of(q, stream)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError(f"q and k must be [B, S, H, D], got {tuple(q.shape)}, {tuple(k.shape)}")
    B, Sq, H, D = shape = q.shape
    Sk, Hk = k.shape[1], k.shape[2]
    if max(B, H, Hk) > 0x7FFFFFFF:
        raise ValueError(f"batch and heads must be below 2^31, got {B}, {H}, {Hk}")
    qp, qb, qr = _head_rows("q", q, shape, dev)
    kp, kb, kr = _head_rows("k", k, (B, Sk, Hk, D), dev)
    vp, vb, vr = _head_rows("v", v, (B, Sk, Hk, D), dev)
    lp = mp = None
    mb = 0
    if lengths is not None:
        if lengths.shape != (B,) or lengths.dtype != torch.int32 or lengths.get_device() != dev \
                or not lengths.is_contiguous():
            raise ValueError(f"lengths must be contiguous int32 [{B}] on cuda:{dev}, got "
                             f"{lengths.dtype} {tuple(lengths.shape)} on {lengths.device}")
        lp = lengths.data_ptr()
    if mask is not None:
        if mask.shape != (B, Sk) or mask.dtype not in (torch.bool, torch.uint8) \
                or mask.get_device() != dev or (mask.stride(1) != 1 and Sk > 1):
            raise ValueError(f"mask must be bool or uint8 [{B}, {Sk}] on cuda:{dev} with its keys "
                             f"adjacent, got {mask.dtype} {tuple(mask.shape)} on {mask.device}")
        mp, mb = mask.data_ptr(), mask.stride(0) if B > 1 else 0
    scale = _softmax_scale(scale)
    if out is None:
        out = _allocate(stream, torch.empty, shape, dtype=torch.bfloat16, device=q.device)
    op, ob, orow = _head_rows("out", out, shape, dev)
    rc = lib.flux_cross_attention(qp, qb, qr, kp, kb, kr, vp, vb, vr, lp, mp, mb, B, Sq, Sk, H, Hk,
                                  D, scale, op, ob, orow, _status_pointer(lib, status, dev),
                                  handle)
    if rc != 0:
        raise FluxError("flux_cross_attention", rc, lib)
    return out


def _status_pointer(lib, status, dev):
    """A caller's status word (int32 [1]), or the device's own."""
    import torch

    if status is None:
        return _own_words.get(dev) or _own_status(lib, dev)
    if status.dtype != torch.int32 or status.numel() < 1 or status.get_device() != dev:
        raise ValueError(f"status must hold one int32 on cuda:{dev}")
    return status.data_ptr()


_own_words = {}  # address of the library's own status word, by device


def _own_status(lib, dev):
    """The library's own status word on `dev`, the current device."""
    if dev not in _own_words:
        word = ctypes.c_void_p()
        rc = lib.flux_status_word(ctypes.byref(word))
        if rc != 0:
            raise FluxError("flux_status_word", rc, lib)
        _own_words[dev] = word.value
        if lib is _compiled_lib:
            _compiled.own_word(dev, word.value)
    return _own_words[dev]


def take_status(stream=None) -> int:
    """Synchronise and return the current device's own status word, which calls
    without ``status`` report to (0, or FLUX_ERR_DEVICE_TIMEOUT if a bounded wait
    of one of them ran out since it was last taken); clears it."""
    lib = load()
    return int(lib.flux_take_status(_stream_handle(stream)))


def query_status(workspace, stream=None) -> int:
    """Synchronise and return the device status word of a call's workspace."""
    lib = load()
    return int(lib.flux_query_status(_ptr(workspace), _stream_handle(stream)))

"""DeepSeek Sparse Attention (DSA) forward pass on B200 (sm_100a).

Thin Python binding over the C ABI of ``libdsa.so`` (declared in
``include/dsa.h``).  Functions carry the C names without the ``dsa_`` prefix and
only marshal arguments: tensors must already be on the GPU, with the dtypes and
shapes the header documents; every step of the computation runs in the
library's CUDA kernels.  PyTorch supplies device memory and streams.

Equations (DeepSeek-V3.2 technical-report summary, section "DSA: внимание
только к важному"):
    I[t,s] = sum_j w[t,j] ReLU(q_I[t,j] . k_I[s])                 (lightning indexer)
    u_t    = Attn(h_t, {c_s : I[t,s] in Top-k(I[t,:])}), k = 2048  (selection + MQA attention)
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "DSAError", "lib", "lib_path", "indexer_scores", "topk", "indexer_topk", "sparse_attn", "sparse_attn_noalloc",
    "forward", "indexer_kl_loss", "indexer_kl_loss_selected",
    "norm_rope", "norm_rope_bwd", "kv4_cache", "kv4_write", "kv4_read", "sparse_attn_kv4", "forward_kv4",
    "window_attn",
    "workspace_size", "workspace_size_args", "status_string", "device_status", "selftest_wait_timeout", "version",
    "OP_TOPK", "OP_SPARSE_ATTN", "OP_FORWARD", "OP_INDEXER_TOPK", "OP_FORWARD_LOWMEM", "OP_WINDOW_ATTN",
    "OP_SPARSE_ATTN_KV4", "OP_FORWARD_KV4",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libdsa.so")

OP_TOPK, OP_SPARSE_ATTN, OP_FORWARD, OP_INDEXER_TOPK, OP_FORWARD_LOWMEM, OP_WINDOW_ATTN = 0, 1, 2, 3, 4, 5
OP_SPARSE_ATTN_KV4, OP_FORWARD_KV4 = 6, 7
_STATUS = {0: "DSA_OK", 1: "DSA_ERR_INVALID_ARG", 2: "DSA_ERR_UNSUPPORTED", 3: "DSA_ERR_WORKSPACE",
           4: "DSA_ERR_CUDA", 5: "DSA_ERR_TIMEOUT"}


class DSAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


class IndexerArgs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Lq", ctypes.c_int), ("Lk", ctypes.c_int), ("q_offset", ctypes.c_int),
                ("H_I", ctypes.c_int), ("d_I", ctypes.c_int),
                ("q_I", ctypes.c_void_p), ("q_scale", ctypes.c_void_p), ("w", ctypes.c_void_p),
                ("k_I", ctypes.c_void_p), ("k_scale", ctypes.c_void_p)]


class AttnArgs(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int), ("d_qk", ctypes.c_int), ("d_v", ctypes.c_int), ("scale", ctypes.c_float),
                ("q", ctypes.c_void_p), ("kv", ctypes.c_void_p)]


class NormRopeArgs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("L", ctypes.c_int), ("H", ctypes.c_int), ("D", ctypes.c_int),
                ("stride_b", ctypes.c_int64), ("stride_l", ctypes.c_int64), ("stride_h", ctypes.c_int64),
                ("x", ctypes.c_void_p), ("norm", ctypes.c_int), ("norm_dim", ctypes.c_int), ("eps", ctypes.c_float),
                ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("weight_bf16", ctypes.c_int),
                ("rot_start", ctypes.c_int), ("n_freq", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("inv_freq", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("q_offset", ctypes.c_int)]


class Kv4Cache(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Lk", ctypes.c_int), ("d_qk", ctypes.c_int), ("d_v", ctypes.c_int),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("tail", ctypes.c_void_p)]


class Kv4AttnArgs(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int), ("d_qk", ctypes.c_int), ("d_v", ctypes.c_int), ("scale", ctypes.c_float),
                ("q", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("tail", ctypes.c_void_p)]


_lib = None


def lib():
    """The loaded libdsa.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise ImportError(f"libdsa.so not built at {lib_path}; run python -m sparse_attention_19_b200.build")
        L = ctypes.CDLL(lib_path)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.dsa_indexer_scores.argtypes = [ctypes.POINTER(IndexerArgs), P, P]
        L.dsa_topk.argtypes = [P, I, I, I, I, I, P, P, Z, P]
        L.dsa_sparse_attn.argtypes = [ctypes.POINTER(AttnArgs), I, I, I, P, I, P, P, P, Z, P]
        L.dsa_sparse_attn_noalloc.argtypes = [ctypes.POINTER(AttnArgs), I, I, I, P, I, P, P, P]
        L.dsa_forward.argtypes = [ctypes.POINTER(IndexerArgs), ctypes.POINTER(AttnArgs), I, P, P, P, P, Z, P]
        L.dsa_forward_timed.argtypes = [ctypes.POINTER(IndexerArgs), ctypes.POINTER(AttnArgs), I, P, P, P, P, P, Z,
                                        P, ctypes.POINTER(ctypes.c_void_p)]
        L.dsa_indexer_topk.argtypes = [ctypes.POINTER(IndexerArgs), I, P, P, P, Z, P]
        L.dsa_indexer_kl_loss.argtypes = [ctypes.POINTER(AttnArgs), I, I, I, P, I, P, P, P, P, P]
        L.dsa_indexer_kl_loss_selected.argtypes = [ctypes.POINTER(AttnArgs), I, I, I, P, I, P, P, P, P, P]
        L.dsa_norm_rope.argtypes = [ctypes.POINTER(NormRopeArgs), P, P, P]
        L.dsa_norm_rope_bwd.argtypes = [ctypes.POINTER(NormRopeArgs), P, P, P, P, P, Z, P]
        L.dsa_norm_rope_bwd_workspace.argtypes = [ctypes.POINTER(NormRopeArgs)]
        L.dsa_norm_rope_bwd_workspace.restype = ctypes.c_size_t
        L.dsa_kv4_write.argtypes = [ctypes.POINTER(Kv4Cache), P, I, P, I, P]
        L.dsa_kv4_read.argtypes = [ctypes.POINTER(Kv4Cache), P, I, P, I, P]
        L.dsa_sparse_attn_kv4.argtypes = [ctypes.POINTER(Kv4AttnArgs), I, I, I, P, I, P, P, P, Z, P]
        L.dsa_forward_kv4.argtypes = [ctypes.POINTER(IndexerArgs), ctypes.POINTER(Kv4AttnArgs), I, P, P, P, P, P, Z, P]
        L.dsa_window_attn.argtypes = [ctypes.POINTER(AttnArgs), I, I, I, I, P, I, I, P, P, P, Z, P]
        L.dsa_workspace_size.argtypes = [I, I, I, I, I, I, I]
        L.dsa_workspace_size.restype = ctypes.c_size_t
        L.dsa_workspace_size_args.argtypes = [I, ctypes.POINTER(IndexerArgs), I, I, I]
        L.dsa_workspace_size_args.restype = ctypes.c_size_t
        L.dsa_status_string.argtypes = [I]
        L.dsa_status_string.restype = ctypes.c_char_p
        L.dsa_device_status.argtypes = [I]
        L.dsa_selftest_wait_timeout.argtypes = [ctypes.c_uint32, P]
        for f in ("dsa_indexer_scores", "dsa_topk", "dsa_indexer_topk", "dsa_sparse_attn", "dsa_sparse_attn_noalloc",
                  "dsa_forward", "dsa_forward_timed", "dsa_indexer_kl_loss", "dsa_indexer_kl_loss_selected",
                  "dsa_norm_rope", "dsa_norm_rope_bwd", "dsa_kv4_write", "dsa_kv4_read",
                  "dsa_sparse_attn_kv4", "dsa_forward_kv4", "dsa_window_attn",
                  "dsa_device_status",
                  "dsa_selftest_wait_timeout", "dsa_version"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(status: int) -> str:
    try:
        return lib().dsa_status_string(int(status)).decode()
    except ImportError:
        return _STATUS.get(int(status), f"status {status}")


def version() -> int:
    return int(lib().dsa_version())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(rc: int, where: str):
    if rc != 0:
        raise DSAError(rc, where)


def _need(t, dtype, shape, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def _u8(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _indexer_args(q_I, q_scale, w, k_I, k_scale, q_offset):
    q_I, k_I = _u8(q_I), _u8(k_I)
    B, Lq, H_I, d_I = q_I.shape
    Lk = k_I.shape[1]
    _need(q_I, torch.uint8, (B, Lq, H_I, d_I), "q_I")
    _need(w, torch.bfloat16, (B, Lq, H_I), "w")
    _need(k_I, torch.uint8, (B, Lk, d_I), "k_I")
    if q_scale is not None:
        _need(q_scale, torch.float32, (B, Lq), "q_scale")
    if k_scale is not None:
        _need(k_scale, torch.float32, (B, Lk), "k_scale")
    return IndexerArgs(B, Lq, Lk, int(q_offset), H_I, d_I, _ptr(q_I), _ptr(q_scale), _ptr(w), _ptr(k_I),
                       _ptr(k_scale))


def _attn_args(q, kv, d_v, scale):
    B, Lq, H, D = q.shape
    _need(q, torch.bfloat16, (B, Lq, H, D), "q")
    _need(kv, torch.bfloat16, (B, kv.shape[1], D), "kv")
    return AttnArgs(H, D, int(d_v), float(scale), _ptr(q), _ptr(kv))


def workspace_size(op: int, B: int, Lq: int, Lk: int, k: int, H: int, d_v: int) -> int:
    return int(lib().dsa_workspace_size(int(op), B, Lq, Lk, k, H, d_v))


def workspace_size_args(op: int, ia: "IndexerArgs", k: int, H: int = 0, d_v: int = 0) -> int:
    """Exact workspace bytes of `op` for these indexer arguments (dsa_workspace_size_args)."""
    return int(lib().dsa_workspace_size_args(int(op), ctypes.byref(ia), int(k), int(H), int(d_v)))


def indexer_scores(q_I, q_scale, w, k_I, k_scale, q_offset=0, scores=None, stream=None):
    """fp32 [B, Lq, Lk] indexer scores, -inf above the causal boundary."""
    a = _indexer_args(q_I, q_scale, w, k_I, k_scale, q_offset)
    if scores is None:
        scores = torch.empty(a.B, a.Lq, a.Lk, dtype=torch.float32, device=w.device)
    _need(scores, torch.float32, (a.B, a.Lq, a.Lk), "scores")
    _check(lib().dsa_indexer_scores(ctypes.byref(a), _ptr(scores), _stream(stream)), "dsa_indexer_scores")
    return scores


def topk(scores, k, q_offset=0, indices=None, workspace=None, stream=None):
    """int32 [B, Lq, k] selected positions (ascending, -1 padded)."""
    B, Lq, Lk = scores.shape
    _need(scores, torch.float32, (B, Lq, Lk), "scores")
    if indices is None:
        indices = torch.empty(B, Lq, k, dtype=torch.int32, device=scores.device)
    _need(indices, torch.int32, (B, Lq, k), "indices")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().dsa_topk(_ptr(scores), B, Lq, Lk, int(q_offset), int(k), _ptr(indices), _ptr(workspace),
                          ws_bytes, _stream(stream)), "dsa_topk")
    return indices


def indexer_topk(q_I, q_scale, w, k_I, k_scale, k, q_offset=0, indices=None, sel_scores=None,
                 want_scores=True, workspace=None, stream=None):
    """Indexer with the top-k fused into it (no score matrix is written).

    Returns (indices int32 [B, Lq, k] ascending, -1 padded; sel_scores fp32 [B, Lq, k]
    or None: the score of each selected position, -inf on padding)."""
    a = _indexer_args(q_I, q_scale, w, k_I, k_scale, q_offset)
    dev = w.device
    if indices is None:
        indices = torch.empty(a.B, a.Lq, k, dtype=torch.int32, device=dev)
    _need(indices, torch.int32, (a.B, a.Lq, k), "indices")
    if sel_scores is None and want_scores:
        sel_scores = torch.empty(a.B, a.Lq, k, dtype=torch.float32, device=dev)
    if sel_scores is not None:
        _need(sel_scores, torch.float32, (a.B, a.Lq, k), "sel_scores")
    need = workspace_size_args(OP_INDEXER_TOPK, a, k)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().dsa_indexer_topk(ctypes.byref(a), int(k), _ptr(indices), _ptr(sel_scores), _ptr(workspace),
                                  nbytes, _stream(stream)), "dsa_indexer_topk")
    return indices, sel_scores


def _workspace(op, B, Lq, Lk, k, H, d_v, device, workspace, ia=None):
    need = workspace_size_args(op, ia, k, H, d_v) if ia is not None else workspace_size(op, B, Lq, Lk, k, H, d_v)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return workspace, nbytes


def sparse_attn(q, kv, indices, d_v, scale, out=None, lse=None, want_lse=True, workspace=None, stream=None):
    """bf16 [B, Lq, H, d_v] attention over the selected latent rows (+ fp32 lse [B, Lq, H])."""
    a = _attn_args(q, kv, d_v, scale)
    B, Lq, H, _ = q.shape
    Lk = kv.shape[1]
    k = indices.shape[-1]
    _need(indices, torch.int32, (B, Lq, k), "indices")
    if out is None:
        out = torch.empty(B, Lq, H, d_v, dtype=torch.bfloat16, device=q.device)
    _need(out, torch.bfloat16, (B, Lq, H, d_v), "out")
    if lse is None and want_lse:
        lse = torch.empty(B, Lq, H, dtype=torch.float32, device=q.device)
    workspace, nbytes = _workspace(OP_SPARSE_ATTN, B, Lq, Lk, k, H, d_v, q.device, workspace)
    _check(lib().dsa_sparse_attn(ctypes.byref(a), B, Lq, Lk, _ptr(indices), k, _ptr(out), _ptr(lse),
                                 _ptr(workspace), nbytes, _stream(stream)), "dsa_sparse_attn")
    return out, lse


NOALLOC_SCRATCH_BYTES = 64 << 20   # DSA_NOALLOC_SCRATCH_BYTES


def sparse_attn_noalloc(q, kv, indices, d_v, scale, out, lse=None, stream=None):
    """sparse_attn into caller-provided `out` (and `lse`), with no device allocation:
    the split-k partials use the library's fixed scratch array (dsa_sparse_attn_noalloc)."""
    a = _attn_args(q, kv, d_v, scale)
    B, Lq, H, _ = q.shape
    Lk = kv.shape[1]
    k = indices.shape[-1]
    _need(indices, torch.int32, (B, Lq, k), "indices")
    _need(out, torch.bfloat16, (B, Lq, H, d_v), "out")
    if lse is not None:
        _need(lse, torch.float32, (B, Lq, H), "lse")
    _check(lib().dsa_sparse_attn_noalloc(ctypes.byref(a), B, Lq, Lk, _ptr(indices), k, _ptr(out), _ptr(lse),
                                         _stream(stream)), "dsa_sparse_attn_noalloc")
    return out, lse


def forward(q_I, q_scale, w, k_I, k_scale, q, kv, k, d_v, scale, q_offset=0, indices=None, out=None,
            lse=None, want_lse=True, workspace=None, stream=None, stage_events=None, sel_scores=None,
            low_memory=False):
    """Indexer -> top-k -> sparse attention.  Returns (indices, out, lse).

    The selection is staged (score matrix in the workspace, then the top-k
    kernel; the faster path) unless ``low_memory`` is set or the given
    ``workspace`` is too small for the score matrix, in which case it is fused
    into the indexer (dsa_indexer_topk).  Both give identical results.
    ``stage_events``: optional four torch.cuda.Event objects, recorded on the
    stream before the indexer, after the indexer, after the top-k (the same
    point when fused) and after the attention.  ``sel_scores``: optional fp32
    [B, Lq, k] tensor that receives the indexer score of every selected position.
    """
    ia = _indexer_args(q_I, q_scale, w, k_I, k_scale, q_offset)
    aa = _attn_args(q, kv, d_v, scale)
    B, Lq, Lk, H = ia.B, ia.Lq, ia.Lk, aa.H
    if indices is None:
        indices = torch.empty(B, Lq, k, dtype=torch.int32, device=q.device)
    _need(indices, torch.int32, (B, Lq, k), "indices")
    if out is None:
        out = torch.empty(B, Lq, H, d_v, dtype=torch.bfloat16, device=q.device)
    _need(out, torch.bfloat16, (B, Lq, H, d_v), "out")
    if lse is None and want_lse:
        lse = torch.empty(B, Lq, H, dtype=torch.float32, device=q.device)
    if sel_scores is not None:
        _need(sel_scores, torch.float32, (B, Lq, k), "sel_scores")
    workspace, nbytes = _workspace(OP_FORWARD_LOWMEM if low_memory else OP_FORWARD, B, Lq, Lk, k, H, d_v,
                                   q.device, workspace, ia=ia)
    ev = None
    if stage_events is not None:
        if len(stage_events) != 4:
            raise ValueError("stage_events needs four events")
        for e in stage_events:          # torch creates the CUDA event on first use
            if not e.cuda_event:
                e.record(stream if stream is not None else torch.cuda.current_stream())
        ev = (ctypes.c_void_p * 4)(*[ctypes.c_void_p(e.cuda_event) for e in stage_events])
    _check(lib().dsa_forward_timed(ctypes.byref(ia), ctypes.byref(aa), int(k), _ptr(indices), _ptr(sel_scores),
                                   _ptr(out), _ptr(lse), _ptr(workspace), nbytes, _stream(stream), ev),
           "dsa_forward")
    return indices, out, lse


def indexer_kl_loss(q, kv, indices, lse, scores, d_v, scale, target=None, want_target=True, kl=None,
                    stream=None):
    """Forward of the indexer's training loss over the selected positions.

    Target p = the attention probabilities (from ``lse`` of sparse_attn on the same
    selection) summed over the heads and L1-normalised; loss per row =
    D_KL(p || softmax over the selected positions of ``scores``).  Returns
    (target fp32 [B, Lq, k] or None, kl fp32 [B, Lq]).
    """
    a = _attn_args(q, kv, d_v, scale)
    B, Lq, H, _ = q.shape
    Lk = kv.shape[1]
    k = indices.shape[-1]
    _need(indices, torch.int32, (B, Lq, k), "indices")
    _need(lse, torch.float32, (B, Lq, H), "lse")
    _need(scores, torch.float32, (B, Lq, Lk), "scores")
    if target is None and want_target:
        target = torch.empty(B, Lq, k, dtype=torch.float32, device=q.device)
    if target is not None:
        _need(target, torch.float32, (B, Lq, k), "target")
    if kl is None:
        kl = torch.empty(B, Lq, dtype=torch.float32, device=q.device)
    _need(kl, torch.float32, (B, Lq), "kl")
    _check(lib().dsa_indexer_kl_loss(ctypes.byref(a), B, Lq, Lk, _ptr(indices), k, _ptr(lse), _ptr(scores),
                                     _ptr(target), _ptr(kl), _stream(stream)), "dsa_indexer_kl_loss")
    return target, kl


def indexer_kl_loss_selected(q, kv, indices, lse, sel_scores, d_v, scale, target=None, want_target=True, kl=None,
                             stream=None):
    """indexer_kl_loss with the scores given per index slot (fp32 [B, Lq, k], as
    returned by indexer_topk or forward(sel_scores=...)) instead of a full matrix."""
    a = _attn_args(q, kv, d_v, scale)
    B, Lq, H, _ = q.shape
    Lk = kv.shape[1]
    k = indices.shape[-1]
    _need(indices, torch.int32, (B, Lq, k), "indices")
    _need(lse, torch.float32, (B, Lq, H), "lse")
    _need(sel_scores, torch.float32, (B, Lq, k), "sel_scores")
    if target is None and want_target:
        target = torch.empty(B, Lq, k, dtype=torch.float32, device=q.device)
    if target is not None:
        _need(target, torch.float32, (B, Lq, k), "target")
    if kl is None:
        kl = torch.empty(B, Lq, dtype=torch.float32, device=q.device)
    _need(kl, torch.float32, (B, Lq), "kl")
    _check(lib().dsa_indexer_kl_loss_selected(ctypes.byref(a), B, Lq, Lk, _ptr(indices), k, _ptr(lse),
                                              _ptr(sel_scores), _ptr(target), _ptr(kl), _stream(stream)),
           "dsa_indexer_kl_loss_selected")
    return target, kl


def _need_at(t, dtype, shape, name, device):
    """_need, and on the same device as the call's other tensors."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    _need(t, dtype, shape, name)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _int32(v, name):
    """v as an int that the C side's 32 bits hold (ctypes would wrap it silently)."""
    v = int(v)
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{name} {v} does not fit 32 bits")
    return v


def _on(device, stream, call, *args):
    """call(stream handle, *args) with `device` current, and with what it allocates belonging to
    the stream that it launches on (a workspace freed on return is then reused in that
    stream's order)."""
    if stream is None and device.index == torch.cuda.current_device():
        return call(torch._C._cuda_getCurrentRawStream(device.index), *args)   # an integer: a Stream object costs 3 us
    if stream is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.device(device):
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(device)):
            return call(torch.cuda.current_stream().cuda_stream, *args)


def _need_workspace(ws, device):
    if ws is not None and (not isinstance(ws, torch.Tensor) or ws.device != device or not ws.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {device}")


def _like(t, dtype, shape, device):
    """torch.empty of this shape and type; from a contiguous tensor of the same shape where
    there is one (half the host time)."""
    if t is not None and t.shape == shape and t.is_contiguous():
        return torch.empty_like(t, dtype=dtype)
    return torch.empty(shape, dtype=dtype, device=device)


_NORMS = {None: 0, "rms": 1, "layer": 2}


def _norm_rope_args(x, inv_freq, weight, bias, norm, norm_dim, eps, rot_start, interleaved, positions, q_offset):
    rot_start, q_offset = _int32(rot_start, "rot_start"), _int32(q_offset, "q_offset")
    if norm_dim is not None:
        norm_dim = _int32(norm_dim, "norm_dim")
    if not isinstance(x, torch.Tensor) or x.dtype != torch.bfloat16:
        raise TypeError("x must be a bfloat16 torch.Tensor")
    if x.dim() != 4:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected [B, L, H, D]")
    if not x.is_cuda or (x.stride(3) != 1 and x.shape[3] > 1):
        raise ValueError("x must be a CUDA tensor with contiguous columns")
    if norm not in _NORMS:
        raise ValueError(f"norm {norm!r}: expected None, 'rms' or 'layer'")
    dev = x.device
    B, L, H, D = x.shape
    w_ptr = b_ptr = f_ptr = pos_ptr = None
    n_freq = w_bf16 = 0
    if norm is not None:
        norm_dim = D if norm_dim is None else norm_dim
        w_bf16 = isinstance(weight, torch.Tensor) and weight.dtype is torch.bfloat16
        wt = torch.bfloat16 if w_bf16 else torch.float32
        _need_at(weight, wt, (norm_dim,), "weight", dev)
        w_ptr = weight.data_ptr()
        if bias is not None:
            _need_at(bias, wt, (norm_dim,), "bias", dev)
            b_ptr = bias.data_ptr()
    elif weight is not None or bias is not None or norm_dim is not None:
        raise ValueError("weight, bias and norm_dim belong to a norm")
    if inv_freq is not None:
        n_freq = inv_freq.numel()
        _need_at(inv_freq, torch.float32, (n_freq,), "inv_freq", dev)
        f_ptr = inv_freq.data_ptr()
    if positions is not None:
        _need_at(positions, torch.int32, (B, L), "positions", dev)
        pos_ptr = positions.data_ptr()
    sb, sl, sh, _ = x.stride()
    return NormRopeArgs(B, L, H, D, sb, sl, sh, x.data_ptr(), _NORMS[norm], norm_dim or 0, eps, w_ptr, b_ptr, w_bf16,
                        rot_start, n_freq, bool(interleaved), f_ptr, pos_ptr, q_offset)


def norm_rope(x, inv_freq=None, *, weight=None, bias=None, norm=None, norm_dim=None, eps=1e-6, rot_start=0,
              interleaved=False, positions=None, q_offset=0, e4m3=False, out=None, scale=None, stream=None):
    """Norm of each head row of ``x`` (bf16 [B, L, H, D], strides over B, L, H in steps of 8) over its
    leading ``norm_dim`` columns (``norm``: None, "rms" or "layer"; weight and bias fp32 or
    bf16), then the position rotation of columns [rot_start, rot_start + 2F) by the angles
    position * ``inv_freq`` (fp32 [F]; positions int32 [B, L], or q_offset + l).

    Returns bf16 [B, L, H, D]; with ``e4m3`` the pair (float8_e4m3fn [B, L, H, D], fp32
    scale [B, L]) that the indexer takes.  ``out`` must not overlap ``x``.  As everywhere in
    this library, the result carries no autograd graph, whatever ``x`` and ``weight`` ask for:
    norm_rope_bwd is the gradient, called with the result's own gradient.
    """
    a = _norm_rope_args(x, inv_freq, weight, bias, norm, norm_dim, eps, rot_start, interleaved, positions, q_offset)
    dev, shape = x.device, x.shape
    out_t = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    if not e4m3 and scale is not None:
        raise ValueError("scale belongs to the e4m3 output")

    def call(st):
        o, sc = out, scale
        if o is None:
            o = _like(x, out_t, shape, dev)
        else:
            _need_at(o, torch.uint8 if e4m3 and o.dtype == torch.uint8 else out_t, shape, "out", dev)
        if e4m3:
            if sc is None:
                sc = _like(positions, torch.float32, shape[:2], dev)
            else:
                _need_at(sc, torch.float32, shape[:2], "scale", dev)
        _check(lib().dsa_norm_rope(ctypes.byref(a), o.data_ptr(), None if sc is None else sc.data_ptr(), st),
               "dsa_norm_rope")
        return (o, sc) if e4m3 else o

    return _on(dev, stream, call)


def norm_rope_bwd(dy, x, inv_freq=None, *, weight=None, bias=None, norm=None, norm_dim=None, eps=1e-6, rot_start=0,
                  interleaved=False, positions=None, q_offset=0, dx=None, dweight=None, dbias=None, workspace=None,
                  stream=None):
    """Gradient of norm_rope's bf16 output: (dx bf16 [B, L, H, D], dweight fp32 or None,
    dbias fp32 or None) for ``dy`` bf16 [B, L, H, D]; the other arguments as in the forward."""
    if norm is None and (dweight is not None or dbias is not None):
        raise ValueError("dweight and dbias belong to a norm")
    a = _norm_rope_args(x, inv_freq, weight, bias, norm, norm_dim, eps, rot_start, interleaved, positions, q_offset)
    dev, shape = x.device, x.shape
    _need_at(dy, torch.bfloat16, shape, "dy", dev)
    _need_workspace(workspace, dev)

    def call(st):
        gx, gw, gb, ws = dx, dweight, dbias, workspace
        if gx is None:
            gx = torch.empty_like(dy)
        else:
            _need_at(gx, torch.bfloat16, shape, "dx", dev)
        if norm is not None:
            of_w = (a.norm_dim,)
            if gw is None:
                gw = _like(weight, torch.float32, of_w, dev)
            else:
                _need_at(gw, torch.float32, of_w, "dweight", dev)
            if gb is None:
                gb = None if bias is None else _like(bias, torch.float32, of_w, dev)
            else:
                _need_at(gb, torch.float32, of_w, "dbias", dev)
            if ws is None:
                ws = torch.empty(lib().dsa_norm_rope_bwd_workspace(ctypes.byref(a)), dtype=torch.uint8, device=dev)
        nbytes = 0 if ws is None else ws.numel() * ws.element_size()
        _check(lib().dsa_norm_rope_bwd(ctypes.byref(a), dy.data_ptr(), gx.data_ptr(), _ptr(gw), _ptr(gb),
                                       None if ws is None else ws.data_ptr(), nbytes, st), "dsa_norm_rope_bwd")
        return gx, gw, gb

    return _on(dev, stream, call)


def kv4_cache(B, Lk, d_qk, d_v, device="cuda"):
    """An empty 4-bit latent cache: (codes uint8 [B, Lk, d_v/2], scales bf16 [B, Lk, d_v/32],
    tail bf16 [B, Lk, d_qk - d_v]).  Rows that nothing was stored in read as zeros."""
    codes = torch.full((B, Lk, d_v // 2), 0x88, dtype=torch.uint8, device=device)
    scales = torch.zeros(B, Lk, d_v // 32, dtype=torch.bfloat16, device=device)
    return codes, scales, torch.zeros(B, Lk, d_qk - d_v, dtype=torch.bfloat16, device=device)


def _kv4(codes, scales, tail):
    if not isinstance(codes, torch.Tensor) or codes.dim() != 3 or not codes.is_cuda:
        raise ValueError("codes must be a CUDA tensor [B, Lk, d_v/2]")
    B, Lk, half = codes.shape
    dev = codes.device
    _need_at(codes, torch.uint8, (B, Lk, half), "codes", dev)
    _need_at(scales, torch.bfloat16, (B, Lk, half // 16), "scales", dev)
    _need_at(tail, torch.bfloat16, (B, Lk, tail.shape[-1]), "tail", dev)
    return Kv4Cache(B, Lk, 2 * half + tail.shape[-1], 2 * half, codes.data_ptr(), scales.data_ptr(), tail.data_ptr())


def kv4_write(kv, codes, scales, tail, start=None, offset=0, stream=None):
    """Stores latent rows ``kv`` (bf16 [B, L, d_qk]) in rows first .. first + L - 1 of each
    sequence of the 4-bit cache; first is ``start`` (int32 [B]) or ``offset``.  Rows outside
    the cache are not stored; the cache's other rows stay as they were."""
    offset = _int32(offset, "offset")
    c = _kv4(codes, scales, tail)
    dev = codes.device
    L = kv.shape[1]
    _need_at(kv, torch.bfloat16, (c.B, L, c.d_qk), "kv", dev)
    if start is not None:
        _need_at(start, torch.int32, (c.B,), "start", dev)
    _on(dev, stream, _kv4_write, c, kv, L, None if start is None else start.data_ptr(), offset)


def _kv4_write(st, c, kv, L, start, offset):
    rc = lib().dsa_kv4_write(ctypes.byref(c), kv.data_ptr(), L, start, offset, st)
    if rc:
        raise DSAError(rc, "dsa_kv4_write")


def kv4_read(codes, scales, tail, L, start=None, offset=0, kv=None, stream=None):
    """bf16 [B, L, d_qk]: rows first .. first + L - 1 of each sequence as the values the
    4-bit cache holds (rows outside the cache: zeros)."""
    L, offset = _int32(L, "L"), _int32(offset, "offset")
    c = _kv4(codes, scales, tail)
    dev = codes.device
    if start is not None:
        _need_at(start, torch.int32, (c.B,), "start", dev)

    def call(st):
        o = kv
        if o is None:
            o = tail.new_empty((c.B, L, c.d_qk))
        else:
            _need_at(o, torch.bfloat16, (c.B, L, c.d_qk), "kv", dev)
        _check(lib().dsa_kv4_read(ctypes.byref(c), o.data_ptr(), L, None if start is None else start.data_ptr(),
                                  offset, st), "dsa_kv4_read")
        return o

    return _on(dev, stream, call)


def _kv4_attn_args(q, codes, scales, tail, scale):
    c = _kv4(codes, scales, tail)
    _, Lq, H, _ = q.shape
    _need_at(q, torch.bfloat16, (c.B, Lq, H, c.d_qk), "q", codes.device)
    return c, Kv4AttnArgs(H, c.d_qk, c.d_v, scale, q.data_ptr(), c.codes, c.scales, c.tail)


def _attn_outputs(q, d_v, out, lse, want_lse):
    B, Lq, H, _ = q.shape
    if out is None:
        out = q.new_empty((B, Lq, H, d_v))
    else:
        _need_at(out, torch.bfloat16, (B, Lq, H, d_v), "out", q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, Lq, H), dtype=torch.float32, device=q.device)
    elif lse is not None:
        _need_at(lse, torch.float32, (B, Lq, H), "lse", q.device)
    return out, lse


def sparse_attn_kv4(q, codes, scales, tail, indices, scale, out=None, lse=None, want_lse=True, workspace=None,
                    stream=None, low_memory=False):
    """sparse_attn over the rows of a 4-bit cache (kv4_cache): bf16 [B, Lq, H, d_v] and fp32
    lse [B, Lq, H].  It reads 416 bytes a row instead of 1152 and takes about as long.  Rows
    that ``indices`` does not name may hold anything.  Without a
    ``workspace`` of the caller's, a prefill chunk takes one with room for the unpacked rows
    (OP_SPARSE_ATTN_KV4, 2.8 times the cache); with ``low_memory`` it takes OP_SPARSE_ATTN bytes,
    the least that a caller may give, and is slower there.  The result is the same."""
    c, a = _kv4_attn_args(q, codes, scales, tail, scale)
    dev, Lq, k = q.device, q.shape[1], indices.shape[-1]
    _need_at(indices, torch.int32, (c.B, Lq, k), "indices", dev)
    _need_workspace(workspace, dev)

    def call(st):
        o, l = _attn_outputs(q, c.d_v, out, lse, want_lse)
        ws, nbytes = _workspace(OP_SPARSE_ATTN if low_memory else OP_SPARSE_ATTN_KV4, c.B, Lq, c.Lk, k, a.H, c.d_v,
                                dev, workspace)
        _check(lib().dsa_sparse_attn_kv4(ctypes.byref(a), c.B, Lq, c.Lk, indices.data_ptr(), k, o.data_ptr(), _ptr(l),
                                         _ptr(ws), nbytes, st), "dsa_sparse_attn_kv4")
        return o, l

    return _on(dev, stream, call)


def forward_kv4(q_I, q_scale, w, k_I, k_scale, q, codes, scales, tail, k, scale, q_offset=0, indices=None, out=None,
                lse=None, want_lse=True, workspace=None, stream=None, sel_scores=None, low_memory=False):
    """forward with the latent rows in a 4-bit cache.  Returns (indices, out, lse).  With
    ``low_memory`` neither scores nor unpacked rows are held (sparse_attn_kv4)."""
    k, q_offset = _int32(k, "k"), _int32(q_offset, "q_offset")
    c, a = _kv4_attn_args(q, codes, scales, tail, scale)
    dev = q.device
    ia = _indexer_args(q_I, q_scale, w, k_I, k_scale, q_offset)
    if (ia.B, ia.Lq, ia.Lk) != (c.B, q.shape[1], c.Lk):
        raise ValueError(f"the indexer's B, Lq, Lk {(ia.B, ia.Lq, ia.Lk)} differ from the attention's "
                         f"{(c.B, q.shape[1], c.Lk)}")
    if any(t is not None and t.device != dev for t in (q_I, q_scale, w, k_I, k_scale)):
        raise ValueError(f"the indexer's tensors must be on {dev}")
    _need_workspace(workspace, dev)
    if sel_scores is not None:
        _need_at(sel_scores, torch.float32, (ia.B, ia.Lq, k), "sel_scores", dev)

    def call(st):
        i = torch.empty(ia.B, ia.Lq, k, dtype=torch.int32, device=dev) if indices is None else indices
        _need_at(i, torch.int32, (ia.B, ia.Lq, k), "indices", dev)
        o, l = _attn_outputs(q, c.d_v, out, lse, want_lse)
        ws, nbytes = _workspace(OP_FORWARD_LOWMEM if low_memory else OP_FORWARD_KV4, ia.B, ia.Lq, ia.Lk, k, a.H,
                                c.d_v, dev, workspace, ia=ia)
        _check(lib().dsa_forward_kv4(ctypes.byref(ia), ctypes.byref(a), k, _ptr(i), _ptr(sel_scores), _ptr(o),
                                     _ptr(l), _ptr(ws), nbytes, st), "dsa_forward_kv4")
        return i, o, l

    return _on(dev, stream, call)


def window_attn(q, kv, d_v, scale, window, sinks=0, q_offset=0, start=None, out=None, lse=None, want_lse=True,
                workspace=None, stream=None):
    """MLA attention where query i of sequence b, at t = (start[b] or q_offset) + i, sees the
    keys (t - window, t] and the first ``sinks`` ones: bf16 [B, Lq, H, d_v] and fp32 lse
    [B, Lq, H].  ``start``: int32 [B], any values; a query that sees nothing gets out = 0 and
    lse = -inf.  Keys that no query sees may hold anything."""
    window = _int32(min(window, 2 ** 31 - 1), "window")     # wider than any sequence: all keys
    sinks = _int32(min(sinks, 2 ** 31 - 1), "sinks")
    q_offset = _int32(q_offset, "q_offset")
    a = _attn_args(q, kv, d_v, scale)
    dev = q.device
    B, Lq, H, _ = q.shape
    Lk = kv.shape[1]
    if kv.device != dev:
        raise ValueError(f"kv is on {kv.device}, expected {dev}")
    if start is not None:
        _need_at(start, torch.int32, (B,), "start", dev)
    _need_workspace(workspace, dev)

    def call(st):
        o, l = _attn_outputs(q, int(d_v), out, lse, want_lse)
        ws, nbytes = _workspace(OP_WINDOW_ATTN, B, Lq, Lk, min(window + sinks, Lk), H, int(d_v), dev, workspace)
        _check(lib().dsa_window_attn(ctypes.byref(a), B, Lq, Lk, q_offset, _ptr(start), window, sinks, _ptr(o),
                                     _ptr(l), _ptr(ws), nbytes, st), "dsa_window_attn")
        return o, l

    return _on(dev, stream, call)


def device_status(clear: bool = True) -> int:
    """0 (DSA_OK) or 5 (DSA_ERR_TIMEOUT): whether a device-side wait gave up.  Synchronises."""
    return int(lib().dsa_device_status(1 if clear else 0))


def selftest_wait_timeout(spin_limit: int = 1 << 16, stream=None) -> int:
    return int(lib().dsa_selftest_wait_timeout(int(spin_limit), _stream(stream)))

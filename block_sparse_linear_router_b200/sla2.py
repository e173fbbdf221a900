"""Thin ctypes binding of libsla2.so (the C ABI in include/sla2.h).

Argument marshalling only: every step of the forward pass runs in the CUDA
kernels of the library. PyTorch provides device memory and streams. There is
no CPU fallback: if the library or a CUDA device is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsla2.so")

STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported shape", 3: "workspace", 4: "CUDA error",
          5: "device wait timed out", 6: "bad page id, length, offset or position"}


class Sla2Error(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: status {code} ({STATUS.get(code, '?')})")
        self.code = code


class Desc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("H", ctypes.c_int), ("N", ctypes.c_int), ("d", ctypes.c_int),
        ("quantize", ctypes.c_int), ("out_dtype", ctypes.c_int),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("status", ctypes.c_void_p),
        ("dbg_scores", ctypes.c_void_p), ("dbg_os", ctypes.c_void_p), ("dbg_ol", ctypes.c_void_p),
        ("dbg_qhat", ctypes.c_void_p), ("dbg_khat", ctypes.c_void_p), ("dbg_vhat", ctypes.c_void_p),
        ("dbg_qscale", ctypes.c_void_p), ("dbg_kscale", ctypes.c_void_p), ("dbg_vscale", ctypes.c_void_p),
        ("dbg_mask", ctypes.c_void_p), ("dbg_idx", ctypes.c_void_p),
        ("stage_events", ctypes.c_void_p),
    ]


class View(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64),
                ("stride_n", ctypes.c_int64)]


class WindowDesc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("N", ctypes.c_int), ("d", ctypes.c_int),
        ("window", ctypes.c_int), ("sinks", ctypes.c_int), ("causal", ctypes.c_int), ("dtype", ctypes.c_int),
        ("scale", ctypes.c_float), ("lens", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t), ("status", ctypes.c_void_p),
    ]


class CacheDesc(ctypes.Structure):
    _fields_ = [
        ("num_pages", ctypes.c_int), ("Hkv", ctypes.c_int), ("page", ctypes.c_int), ("d", ctypes.c_int),
        ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
    ]


class StepDesc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("Hq", ctypes.c_int), ("max_pages", ctypes.c_int),
        ("dtype", ctypes.c_int), ("page_table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p),
        ("cu_new", ctypes.c_void_p), ("status", ctypes.c_void_p),
    ]


STAGE_EVENTS = 5   # [start, router done, linear state done, sparse done, end]


# The exported symbols and their C signatures (checked by the CPU tests).
SIGNATURES = {
    "sla2_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "sla2_topk_count": (ctypes.c_int, [ctypes.c_int, ctypes.c_float]),
    "sla2_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(Desc), ctypes.c_float]),
    "sla2_router": (ctypes.c_int, [ctypes.POINTER(Desc)] + [ctypes.c_void_p] * 4 + [ctypes.c_float]
                    + [ctypes.c_void_p] * 4),
    "sla2_router_soft": (ctypes.c_int, [ctypes.POINTER(Desc)] + [ctypes.c_void_p] * 4
                         + [ctypes.c_float, ctypes.c_float] + [ctypes.c_void_p] * 3),
    "sla2_linear_state": (ctypes.c_int, [ctypes.POINTER(Desc)] + [ctypes.c_void_p] * 8),
    "sla2_forward": (ctypes.c_int, [ctypes.POINTER(Desc)] + [ctypes.c_void_p] * 6 + [ctypes.c_float]
                     + [ctypes.c_void_p] * 2),
    "sla2_workspace_size_heads": (ctypes.c_size_t, [ctypes.POINTER(Desc), ctypes.c_int, ctypes.c_float]),
    "sla2_backward_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(Desc), ctypes.c_float]),
    "sla2_backward": (ctypes.c_int, [ctypes.POINTER(Desc)] + [ctypes.c_void_p] * 6 + [ctypes.c_float]
                      + [ctypes.c_void_p] * 6),
    "sla2_forward_heads": (ctypes.c_int, [ctypes.POINTER(Desc), ctypes.c_int, ctypes.c_int] + [ctypes.c_void_p] * 6
                           + [ctypes.c_float] + [ctypes.c_void_p] * 2),
    "sla2_forward_host_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(Desc), ctypes.c_int, ctypes.c_float]),
    "sla2_forward_host": (ctypes.c_int, [ctypes.POINTER(Desc), ctypes.c_int] + [ctypes.c_void_p] * 6
                          + [ctypes.c_float] + [ctypes.c_void_p] * 2),
    "sla2_window_forward": (ctypes.c_int, [ctypes.POINTER(WindowDesc)] + [ctypes.POINTER(View)] * 4
                            + [ctypes.c_void_p] * 2),
    "sla2_window_backward_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(WindowDesc)]),
    "sla2_window_backward": (ctypes.c_int, [ctypes.POINTER(WindowDesc)] + [ctypes.POINTER(View)] * 4
                             + [ctypes.c_void_p] + [ctypes.POINTER(View)] * 4 + [ctypes.c_void_p]),
    "sla2_cache_append": (ctypes.c_int, [ctypes.POINTER(CacheDesc), ctypes.POINTER(StepDesc)]
                          + [ctypes.POINTER(View)] * 5 + [ctypes.c_void_p] * 2 + [ctypes.c_int] * 3
                          + [ctypes.c_void_p]),
    "sla2_cache_attention_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(CacheDesc), ctypes.POINTER(StepDesc)]),
    "sla2_cache_attention": (ctypes.c_int, [ctypes.POINTER(CacheDesc), ctypes.POINTER(StepDesc)]
                             + [ctypes.POINTER(View)] * 2 + [ctypes.c_int] * 2 + [ctypes.c_float, ctypes.c_void_p,
                                                                                  ctypes.c_size_t, ctypes.c_void_p]),
}

_lib = None


def load_library(path: str = LIB_PATH):
    """Load libsla2.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libsla2.so not built ({path}); run python -m block_sparse_linear_router_b200.build")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    lib.sla2_set_wait_budget_ns.restype = None
    lib.sla2_set_wait_budget_ns.argtypes = [ctypes.c_ulonglong]
    _lib = lib
    return lib


def topk_count(nk: int, frac: float) -> int:
    return load_library().sla2_topk_count(nk, frac)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check_qkv(*ts):
    for t in ts:
        if not t.is_cuda:
            raise ValueError("tensors must be on a CUDA device (no CPU path)")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def make_desc(B, H, N, d, quantize=1, out_dtype=0) -> Desc:
    return Desc(B=B, H=H, N=N, d=d, quantize=quantize, out_dtype=out_dtype)


def workspace_size(B, H, N, d, frac, quantize=1) -> int:
    desc = make_desc(B, H, N, d, quantize)
    return load_library().sla2_workspace_size(ctypes.byref(desc), frac)


def set_wait_budget_ns(ns: int) -> None:
    load_library().sla2_set_wait_budget_ns(int(ns))


@dataclass
class Workspace:
    buf: torch.Tensor

    @staticmethod
    def for_shape(B, H, N, d, frac, quantize=1, device="cuda") -> "Workspace":
        n = workspace_size(B, H, N, d, frac, quantize)
        if n == 0:
            raise Sla2Error(1, "sla2_workspace_size")
        return Workspace(torch.empty(n, dtype=torch.uint8, device=device))


def router(q, k, proj_q, proj_k, frac, workspace: Optional[Workspace] = None, scores=False, stream=None):
    """Mask M_c (uint8 [B,H,nq,nk]), idx (int32 [B,H,nq,k]), colmean (fp32 [B,H,d]) and optionally the fp32 logits."""
    lib = load_library()
    _check_qkv(q, k, proj_q, proj_k)
    B, H, N, d = q.shape
    nq, nk = N // 128, N // 64
    kk = lib.sla2_topk_count(nk, frac)
    ws = workspace or Workspace.for_shape(B, H, N, d, frac, 0, q.device)
    desc = make_desc(B, H, N, d, 0)
    desc.workspace, desc.workspace_bytes = ws.buf.data_ptr(), ws.buf.numel()
    mask = torch.empty(B, H, nq, nk, dtype=torch.uint8, device=q.device)
    idx = torch.empty(B, H, nq, max(kk, 1), dtype=torch.int32, device=q.device)
    cm = torch.empty(B, H, d, dtype=torch.float32, device=q.device)
    sc = torch.empty(B, H, nq, nk, dtype=torch.float32, device=q.device) if scores else None
    if sc is not None:
        desc.dbg_scores = sc.data_ptr()
    r = lib.sla2_router(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(proj_q), _ptr(proj_k), frac,
                        _ptr(mask), _ptr(idx), _ptr(cm), _stream(stream))
    if r != 0:
        raise Sla2Error(r, "sla2_router")
    out = {"mask": mask, "idx": idx, "colmean": cm}
    if sc is not None:
        out["scores"] = sc
    return out


def router_soft(q, k, proj_q, proj_k, frac, tau=0.1, workspace: Optional[Workspace] = None, scores=False,
                stream=None):
    """SoftTop-k mask sigmoid(P_c / tau + lambda) (fp32 [B,H,nq,nk], rows summing to k) and lambda
    (fp32 [B,H,nq]); optionally the fp32 logits."""
    lib = load_library()
    _check_qkv(q, k, proj_q, proj_k)
    B, H, N, d = q.shape
    nq, nk = N // 128, N // 64
    ws = workspace or Workspace.for_shape(B, H, N, d, frac, 0, q.device)
    desc = make_desc(B, H, N, d, 0)
    desc.workspace, desc.workspace_bytes = ws.buf.data_ptr(), ws.buf.numel()
    soft = torch.empty(B, H, nq, nk, dtype=torch.float32, device=q.device)
    lam = torch.empty(B, H, nq, dtype=torch.float32, device=q.device)
    sc = torch.empty(B, H, nq, nk, dtype=torch.float32, device=q.device) if scores else None
    if sc is not None:
        desc.dbg_scores = sc.data_ptr()
    r = lib.sla2_router_soft(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(proj_q), _ptr(proj_k), frac, tau,
                             _ptr(soft), _ptr(lam), _stream(stream))
    if r != 0:
        raise Sla2Error(r, "sla2_router_soft")
    out = {"soft": soft, "lambda": lam}
    if sc is not None:
        out["scores"] = sc
    return out


def linear_state(k, v, colmean, workspace: Optional[Workspace] = None, stream=None):
    """Per key block h_j^T (fp32 [B,H,nk,d(c),d(e)]), z_j, and their sums H_total^T, Z_total, for the
    smoothed keys K - colmean."""
    lib = load_library()
    _check_qkv(k, v, colmean)
    B, H, N, d = k.shape
    nk = N // 64
    ws = workspace or Workspace.for_shape(B, H, N, d, 1.0, 0, k.device)
    desc = make_desc(B, H, N, d, 0)
    desc.workspace, desc.workspace_bytes = ws.buf.data_ptr(), ws.buf.numel()
    dev = k.device
    h = torch.empty(B, H, nk, d, d, dtype=torch.float32, device=dev)
    z = torch.empty(B, H, nk, d, dtype=torch.float32, device=dev)
    Ht = torch.empty(B, H, d, d, dtype=torch.float32, device=dev)
    Zt = torch.empty(B, H, d, dtype=torch.float32, device=dev)
    r = lib.sla2_linear_state(ctypes.byref(desc), _ptr(k), _ptr(v), _ptr(colmean), _ptr(h), _ptr(z), _ptr(Ht),
                              _ptr(Zt), _stream(stream))
    if r != 0:
        raise Sla2Error(r, "sla2_linear_state")
    return {"h": h, "z": z, "Htot": Ht, "Ztot": Zt}


def forward(q, k, v, proj_q, proj_k, alpha, frac, quantize=1, out_dtype=torch.bfloat16,
            workspace: Optional[Workspace] = None, out: Optional[torch.Tensor] = None, debug=False,
            status: Optional[torch.Tensor] = None, stream=None, stage_events=None):
    """The SLA2 forward pass: returns out [B,H,N,d] (and a dict of debug exports when debug=True)."""
    lib = load_library()
    _check_qkv(q, k, v, proj_q, proj_k, alpha)
    B, H, N, d = q.shape
    nq, nk = N // 128, N // 64
    f32 = out_dtype == torch.float32
    ws = workspace or Workspace.for_shape(B, H, N, d, frac, quantize, q.device)
    desc = make_desc(B, H, N, d, quantize, 1 if f32 else 0)
    desc.workspace, desc.workspace_bytes = ws.buf.data_ptr(), ws.buf.numel()
    if out is None:
        out = torch.empty(B, H, N, d, dtype=torch.float32 if f32 else torch.bfloat16, device=q.device)
    if status is not None:
        desc.status = status.data_ptr()
    if stage_events is not None:
        # a ctypes array of STAGE_EVENTS raw cudaEvent_t handles (kept alive by the caller)
        desc.stage_events = ctypes.cast(stage_events, ctypes.c_void_p)
    dbg = {}
    if debug:
        dev = q.device
        kk = lib.sla2_topk_count(nk, frac)
        dbg = {
            "scores": torch.empty(B, H, nq, nk, dtype=torch.float32, device=dev),
            "O_s": torch.empty(B, H, N, d, dtype=torch.float32, device=dev),
            "O_l": torch.empty(B, H, N, d, dtype=torch.float32, device=dev),
            "mask": torch.empty(B, H, nq, nk, dtype=torch.uint8, device=dev),
            "idx": torch.empty(B, H, nq, kk, dtype=torch.int32, device=dev),
        }
        desc.dbg_scores, desc.dbg_os, desc.dbg_ol = (dbg[n].data_ptr() for n in ("scores", "O_s", "O_l"))
        desc.dbg_mask, desc.dbg_idx = dbg["mask"].data_ptr(), dbg["idx"].data_ptr()
        if quantize:
            dbg.update({
                "qhat": torch.empty(B, H, N, d, dtype=torch.int8, device=dev),
                "khat": torch.empty(B, H, N, d, dtype=torch.int8, device=dev),
                "vhatT": torch.empty(B, H, nk, d, 64, dtype=torch.uint8, device=dev),
                "sq": torch.empty(B, H, nq, dtype=torch.float32, device=dev),
                "sk": torch.empty(B, H, nk, dtype=torch.float32, device=dev),
                "sv": torch.empty(B, H, d, dtype=torch.float32, device=dev),
            })
            desc.dbg_qhat, desc.dbg_khat, desc.dbg_vhat = (dbg[n].data_ptr() for n in ("qhat", "khat", "vhatT"))
            desc.dbg_qscale, desc.dbg_kscale, desc.dbg_vscale = (dbg[n].data_ptr() for n in ("sq", "sk", "sv"))
    r = lib.sla2_forward(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(proj_q), _ptr(proj_k), _ptr(alpha),
                         frac, _ptr(out), _stream(stream))
    if r != 0:
        raise Sla2Error(r, "sla2_forward")
    return (out, dbg) if debug else out


def shard_heads(H: int, world_size: int, rank: int):
    """Contiguous head range (h_begin, h_count) of `rank` when H heads are split
    over `world_size` ranks as evenly as possible (the first H % world_size
    ranks take one head more). A rank may get h_count = 0 when world_size > H."""
    if world_size < 1 or not (0 <= rank < world_size) or H < 0:
        raise ValueError("bad head sharding arguments")
    base, extra = divmod(H, world_size)
    h_begin = rank * base + min(rank, extra)
    return h_begin, base + (1 if rank < extra else 0)


def workspace_size_heads(B, H, N, d, h_count, frac, quantize=1) -> int:
    desc = make_desc(B, H, N, d, quantize)
    return load_library().sla2_workspace_size_heads(ctypes.byref(desc), h_count, frac)


def forward_heads(q, k, v, proj_q, proj_k, alpha, frac, h_begin, h_count, out, quantize=1,
                  workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """Heads [h_begin, h_begin + h_count) of the forward pass, written into the full
    output tensor `out` [B,H,N,d] (bf16 or fp32); nothing else of `out` is touched.
    Bit-identical to those heads of forward() on the same full inputs."""
    lib = load_library()
    _check_qkv(q, k, v, proj_q, proj_k, alpha, out)
    B, H, N, d = q.shape
    if out.dtype not in (torch.bfloat16, torch.float32) or tuple(out.shape) != (B, H, N, d):
        raise ValueError("out must be a bf16 or fp32 [B,H,N,d] tensor")
    n = lib.sla2_workspace_size_heads(ctypes.byref(make_desc(B, H, N, d, quantize)), h_count, frac)
    if n == 0:
        raise Sla2Error(1, "sla2_workspace_size_heads")
    ws = workspace if workspace is not None else torch.empty(n, dtype=torch.uint8, device=q.device)
    desc = make_desc(B, H, N, d, quantize, 1 if out.dtype == torch.float32 else 0)
    desc.workspace, desc.workspace_bytes = ws.data_ptr(), ws.numel()
    if status is not None:
        desc.status = status.data_ptr()
    r = lib.sla2_forward_heads(ctypes.byref(desc), h_begin, h_count, _ptr(q), _ptr(k), _ptr(v), _ptr(proj_q),
                               _ptr(proj_k), _ptr(alpha), frac, _ptr(out), _stream(stream))
    if r != 0:
        raise Sla2Error(r, "sla2_forward_heads")
    return out


def forward_host_workspace_size(B, H, N, d, frac, heads_per_group, quantize=1, out_dtype=torch.bfloat16) -> int:
    desc = make_desc(B, H, N, d, quantize, 1 if out_dtype == torch.float32 else 0)
    return load_library().sla2_forward_host_workspace_size(ctypes.byref(desc), heads_per_group, frac)


def forward_host(q, k, v, proj_q, proj_k, alpha, frac, out, heads_per_group=2, quantize=1,
                 workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """The forward pass from HOST tensors to the HOST tensor `out` (bf16 or fp32 [B,H,N,d]),
    with the copies overlapped with the computation head group by head group; the
    workspace is device memory. Returns once enqueued: `out` is complete when `stream`
    (default: the current stream) is, and the host tensors must live until then
    (page-locked tensors let the copies run asynchronously)."""
    lib = load_library()
    for t in (q, k, v, proj_q, proj_k, alpha, out):
        if t.is_cuda:
            raise ValueError("forward_host takes host tensors")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    B, H, N, d = q.shape
    if out.dtype not in (torch.bfloat16, torch.float32) or tuple(out.shape) != (B, H, N, d):
        raise ValueError("out must be a bf16 or fp32 [B,H,N,d] tensor")
    f32 = 1 if out.dtype == torch.float32 else 0
    desc = make_desc(B, H, N, d, quantize, f32)
    n = lib.sla2_forward_host_workspace_size(ctypes.byref(desc), heads_per_group, frac)
    if n == 0:
        raise Sla2Error(1, "sla2_forward_host_workspace_size")
    ws = workspace if workspace is not None else torch.empty(n, dtype=torch.uint8, device="cuda")
    if not ws.is_cuda:
        raise ValueError("the workspace is device memory")
    desc.workspace, desc.workspace_bytes = ws.data_ptr(), ws.numel()
    if status is not None:
        desc.status = status.data_ptr()
    r = lib.sla2_forward_host(ctypes.byref(desc), heads_per_group, _ptr(q), _ptr(k), _ptr(v), _ptr(proj_q),
                              _ptr(proj_k), _ptr(alpha), frac, _ptr(out), _stream(stream))
    if r != 0:
        raise Sla2Error(r, "sla2_forward_host")
    return out


def backward(q, k, v, proj_q, proj_k, alpha, frac, dout, workspace: Optional[torch.Tensor] = None,
             status: Optional[torch.Tensor] = None, stream=None):
    """Gradients of the unquantised forward for the router's mask: (dq, dk, dv) fp32
    [B,H,N,d] and dalpha fp32 [H,nq] (summed over the batch), for dL/dO = dout (fp32)."""
    lib = load_library()
    _check_qkv(q, k, v, proj_q, proj_k, alpha, dout)
    if dout.dtype != torch.float32 or tuple(dout.shape) != tuple(q.shape):
        raise ValueError("dout must be fp32 with the shape of q")
    B, H, N, d = q.shape
    desc = make_desc(B, H, N, d, 0)
    n = lib.sla2_backward_workspace_size(ctypes.byref(desc), frac)
    if n == 0:
        raise Sla2Error(1, "sla2_backward_workspace_size")
    ws = workspace if workspace is not None else torch.empty(n, dtype=torch.uint8, device=q.device)
    desc.workspace, desc.workspace_bytes = ws.data_ptr(), ws.numel()
    if status is not None:
        desc.status = status.data_ptr()
    dq, dk, dv = (torch.empty(B, H, N, d, dtype=torch.float32, device=q.device) for _ in range(3))
    dalpha = torch.empty(H, N // 128, dtype=torch.float32, device=q.device)
    r = lib.sla2_backward(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(proj_q), _ptr(proj_k), _ptr(alpha),
                          frac, _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dalpha), _stream(stream))
    if r != 0:
        raise Sla2Error(r, "sla2_backward")
    return dq, dk, dv, dalpha


# ------------------------------------------------------------------ streaming attention

_DTYPE = {torch.bfloat16: 0, torch.float16: 1}


def _check(ok, what):
    if not ok:
        raise ValueError(what)


def _one_device(first, *others):
    """The index of the CUDA device that all of the tensors (None left out) are on."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device (no CPU path)")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensors must be on one device")
    return dev


def _enqueue(dev, stream, tensors, body):
    """Runs body(raw stream) on `stream` (default: the device's current one), with that device and
    stream current, so that what body allocates belongs to the stream; the caller's tensors are kept
    from reuse until the stream has passed this call."""
    if stream is None and dev == torch.cuda.current_device():
        return body(torch._C._cuda_getCurrentRawStream(dev))
    here = torch.cuda.current_stream(dev)
    if stream is None:
        stream = here
    _check(stream.device.index == dev, "the stream is of another device than the tensors")
    with torch.cuda.stream(stream):
        if stream != here:
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
        return body(stream.cuda_stream)


def _view4(t):
    sb, sh, sn, unit = t.stride()
    if unit != 1:
        raise ValueError("the last dimension must be contiguous")
    return View(t.data_ptr(), sb, sh, sn)


def _view3(t):
    st, sh, unit = t.stride()
    if unit != 1:
        raise ValueError("the last dimension must be contiguous")
    return View(t.data_ptr(), 0, sh, st)


def _status_ok(status):
    _check(status is None or (status.numel() == 1 and status.element_size() == 4), "status must be one 32-bit word")


def _window_desc(q, k, v, window, sinks, causal, scale, lens, status, others):
    qs, ks, dtype = q.shape, k.shape, q.dtype
    if len(qs) != 4 or len(ks) != 4:
        raise ValueError("q, k, v must be [B, H, N, d]")
    B, Hq, N, d = qs
    Hkv = ks[1]
    if ks[0] != B or ks[2] != N or ks[3] != d or v.shape != ks:
        raise ValueError("k and v must be [B, Hkv, N, d] with q's B, N, d")
    if Hkv < 1 or Hq % Hkv:
        raise ValueError("the query heads must be a multiple of the key heads")
    kind = _DTYPE.get(dtype)
    if kind is None or k.dtype != dtype or v.dtype != dtype:
        raise ValueError("q, k, v must be bf16, or fp16")
    for t in others:
        if t is not None and (t.dtype != dtype or t.shape != qs):
            raise ValueError("outputs and gradients have q's type and shape")
    if lens is not None and (lens.dtype != torch.int32 or lens.shape != (B,) or not lens.is_contiguous()):
        raise ValueError("lens must be int32 [B]")
    if not window >= 1:
        raise ValueError("window must be at least 1")
    if not sinks >= 0:
        raise ValueError("sinks must not be negative")
    if status is not None:
        _status_ok(status)
    return WindowDesc(B, Hq, Hkv, N, d, min(window, 0x7fffffff), min(sinks, 0x7fffffff), 1 if causal else 0, kind,
                      d ** -0.5 if scale is None else scale, None if lens is None else lens.data_ptr(), None, 0,
                      None if status is None else status.data_ptr())


def window_forward(q, k, v, window, sinks=0, causal=True, scale=None, lens=None, out: Optional[torch.Tensor] = None,
                   return_lse=False, status: Optional[torch.Tensor] = None, stream=None):
    """Attention through a sliding window with sinks: position i sees key j when i - window < j <= i
    (causal) or |i - j| < window (not causal), and the first `sinks` keys (j <= i where causal).

    q [B,Hq,N,d], k and v [B,Hkv,N,d], bf16 or fp16, d in {64, 128}, any strides that are multiples
    of 8 with a contiguous last dimension; Hq a multiple of Hkv. scale: of the logits, 1/sqrt(d) by
    default. lens: int32 [B] on the device, the sequences' lengths in a padded batch; the rows behind
    them are not seen and come out as zero. Returns out (q's shape, type and layout) and, with
    return_lse, the logarithms of the softmax sums (fp32 [B,Hq,N]) that window_backward takes."""
    desc = _window_desc(q, k, v, window, sinks, causal, scale, lens, status, (out,))
    views = _view4(q), _view4(k), _view4(v)
    to = None if out is None else _view4(out)
    dev = _one_device(q, k, v, lens, out, status)

    def body(raw):
        o = torch.empty_like(q) if out is None else out
        lse = q.new_empty((desc.B, desc.Hq, desc.N), dtype=torch.float32) if return_lse else None
        r = load_library().sla2_window_forward(desc, *views, _view4(o) if to is None else to,
                                               None if lse is None else lse.data_ptr(), raw)
        if r != 0:
            raise Sla2Error(r, "sla2_window_forward")
        return (o, lse) if return_lse else o

    return _enqueue(dev, stream, (q, k, v, lens, out, status), body)


def window_backward(q, k, v, out, lse, dout, window, sinks=0, causal=True, scale=None, lens=None,
                    workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """Gradients (dq, dk, dv), of the inputs' types and shapes, of window_forward for dL/d(out) = dout
    (q's type and shape). out and lse are what window_forward returned for the same arguments; rows
    behind a sequence's length get zero. workspace: device memory of the size
    sla2_window_backward_workspace_size gives, by default allocated here; one call at a time may use it."""
    desc = _window_desc(q, k, v, window, sinks, causal, scale, lens, status, (out, dout))
    _check(lse.dtype == torch.float32 and lse.shape == q.shape[:3] and lse.is_contiguous(), "lse must be fp32 [B, Hq, N]")
    views = _view4(q), _view4(k), _view4(v), _view4(out)
    tdo = _view4(dout)
    dev = _one_device(q, k, v, out, lse, dout, lens, workspace, status)
    lib = load_library()

    def body(raw):
        ws = workspace
        if ws is None:
            n = lib.sla2_window_backward_workspace_size(desc)
            if n == 0:
                raise Sla2Error(1, "sla2_window_backward_workspace_size")
            ws = q.new_empty(n, dtype=torch.uint8)
        desc.workspace, desc.workspace_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        r = lib.sla2_window_backward(desc, *views, lse.data_ptr(), tdo, _view4(dq), _view4(dk), _view4(dv), raw)
        if r != 0:
            raise Sla2Error(r, "sla2_window_backward")
        return dq, dk, dv

    return _enqueue(dev, stream, (q, k, v, out, lse, dout, lens, workspace, status), body)


@dataclass(frozen=True)
class KVCache:
    """A paged cache of keys and values in signed 8-bit codes, one fp32 scale for each page and head:
    codes int8 [num_pages, Hkv, page, d], scales fp32 [num_pages, Hkv]; page in {16, 32, 64, 128}."""
    k_codes: torch.Tensor
    v_codes: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    def __post_init__(self):
        kc, vc, ks, vs = self.k_codes, self.v_codes, self.k_scale, self.v_scale
        _check(kc.dim() == 4 and kc.dtype == torch.int8 and vc.dtype == torch.int8 and vc.shape == kc.shape,
               "codes must be int8 [num_pages, Hkv, page, d]")
        _check(ks.dtype == torch.float32 and vs.dtype == torch.float32 and ks.shape == kc.shape[:2] and vs.shape == ks.shape,
               "scales must be fp32 [num_pages, Hkv]")
        for t in (kc, vc, ks, vs):
            _check(t.is_contiguous(), "tensors must be contiguous")
        n, Hkv, page, d = kc.shape
        object.__setattr__(self, "desc", CacheDesc(num_pages=n, Hkv=Hkv, page=page, d=d, k_codes=kc.data_ptr(),
                                                   v_codes=vc.data_ptr(), k_scale=ks.data_ptr(), v_scale=vs.data_ptr()))

    @staticmethod
    def empty(num_pages: int, Hkv: int, page: int, d: int, device="cuda") -> "KVCache":
        codes = [torch.zeros(num_pages, Hkv, page, d, dtype=torch.int8, device=device) for _ in range(2)]
        scales = [torch.zeros(num_pages, Hkv, dtype=torch.float32, device=device) for _ in range(2)]
        return KVCache(codes[0], codes[1], scales[0], scales[1])


def _step_desc(cache, x, heads, page_table, kv_lens, cu_new, status):
    c, xs, ts = cache.desc, x.shape, page_table.shape
    if len(xs) != 3 or xs[2] != c.d:
        raise ValueError("token arrays must be [T, H, d] with the cache's d")
    kind = _DTYPE.get(x.dtype)
    if kind is None:
        raise ValueError("token arrays must be bf16, or fp16")
    if page_table.dtype != torch.int32 or len(ts) != 2 or not page_table.is_contiguous():
        raise ValueError("page_table must be int32 [B, max_pages]")
    B = ts[0]
    if kv_lens.dtype != torch.int32 or kv_lens.shape != (B,) or not kv_lens.is_contiguous():
        raise ValueError("kv_lens must be int32 [B]")
    if cu_new.dtype != torch.int32 or cu_new.shape != (B + 1,) or not cu_new.is_contiguous():
        raise ValueError("cu_new must be int32 [B + 1]")
    if heads < 1 or heads % c.Hkv:
        raise ValueError("the query heads must be a multiple of the cache's heads")
    if status is not None:
        _status_ok(status)
    return StepDesc(B, xs[0], heads, ts[1], kind, page_table.data_ptr(), kv_lens.data_ptr(), cu_new.data_ptr(),
                    None if status is None else status.data_ptr())


def cache_append(cache: KVCache, k, v, page_table, kv_lens, cu_new,
                 rope: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, interleaved=False,
                 q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """Appends the new tokens of a step to the cache, keys rotated for their positions.

    k, v [T,Hkv,d] (bf16 or fp16): the rows [cu_new[b], cu_new[b+1]) are sequence b's, at the positions
    from kv_lens[b] (the tokens it has in the cache before this call) on. page_table int32
    [B,max_pages], kv_lens int32 [B], cu_new int32 [B+1], on the device; kv_lens is not changed.
    rope: (cos, sin), fp32 [positions, rope_dim/2], rope_dim a multiple of 16 up to d; element i turns
    with i + rope_dim/2, or 2i with 2i + 1 (interleaved). A page's scale grows to the largest value put
    into it, and the codes already there are rounded to the new scale. Given q [T,Hq,d], returns its
    rotated rows (in q_out if given); k_out receives the rotated keys. What is out of range on the
    device (a page id, a position behind the rope's rows, and the sequences from the first bad offset
    on) is left out and reported as 6 in status; rows left out are not written in q_out and k_out."""
    Hq = k.shape[1] if q is None else q.shape[1]
    step = _step_desc(cache, k, Hq, page_table, kv_lens, cu_new, status)
    c = cache.desc
    _check(k.shape[1] == c.Hkv and v.shape == k.shape and v.dtype == k.dtype, "k and v must be [T, Hkv, d] of one type")
    _check(k_out is None or (k_out.shape == k.shape and k_out.dtype == k.dtype), "k_out must be like k")
    _check(q is not None or q_out is None, "q_out without q")
    if q is not None:
        _check(q.shape == (step.T, Hq, c.d) and q.dtype == k.dtype, "q must be [T, Hq, d] of k's type")
        _check(q_out is None or (q_out.shape == q.shape and q_out.dtype == q.dtype), "q_out must be like q")
    tk, tv, tq, tqo, tko = (None if t is None else _view3(t) for t in (k, v, q, q_out, k_out))
    cos, sin = (None, None) if rope is None else rope
    rows = half = 0
    if rope is not None:
        _check(cos.dtype == torch.float32 and cos.dim() == 2 and sin.dtype == cos.dtype and sin.shape == cos.shape
               and cos.is_contiguous() and sin.is_contiguous(), "rope must be two fp32 [positions, rope_dim / 2] tensors")
        rows, half = cos.shape
        _check(half > 0 and half % 8 == 0 and 2 * half <= c.d, "rope_dim must be a multiple of 16, at most d")
    dev = _one_device(k, cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale, v, page_table, kv_lens, cu_new, cos,
                      sin, q, q_out, k_out, status)

    def body(raw):
        o = torch.empty_like(q) if q is not None and q_out is None else q_out
        if step.T == 0:
            if status is not None:
                status.zero_()
            return o
        r = load_library().sla2_cache_append(c, step, tk, tv, tq, _view3(o) if tqo is None and o is not None else tqo, tko,
                                             None if cos is None else cos.data_ptr(),
                                             None if sin is None else sin.data_ptr(), rows, 2 * half,
                                             1 if interleaved else 0, raw)
        if r != 0:
            raise Sla2Error(r, "sla2_cache_append")
        return o

    return _enqueue(dev, stream, (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale, k, v, page_table, kv_lens,
                                  cu_new, cos, sin, q, q_out, k_out, status), body)


def cache_attention_workspace_size(cache: KVCache, T: int, Hq: int, B: int, max_pages: int) -> int:
    """Bytes of workspace that cache_attention takes for T query rows of B sequences."""
    token = ctypes.c_void_p(16)      # stands for the arrays: a size is computed, nothing is read
    step = StepDesc(B=B, T=T, Hq=Hq, max_pages=max_pages, dtype=0, page_table=token, kv_lens=token, cu_new=token)
    return load_library().sla2_cache_attention_workspace_size(cache.desc, step)


def cache_attention(cache: KVCache, q, page_table, kv_lens, cu_new, window: Optional[int] = None, sinks=0, scale=None,
                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream=None):
    """Attention of a step's new tokens over the cache that holds them already: call it after
    cache_append with the same page_table, kv_lens and cu_new.

    q [T,Hq,d] (rotated): row cu_new[b] + i is at position kv_lens[b] + i and sees the keys up to it,
    those of the window (None: all of them) and the first `sinks`. Returns out [T,Hq,d]; rows from
    cu_new[B] on, and those of sequences left out (see cache_append), are left as they are: where out is
    not given they hold whatever was in memory. scale: of the logits, 1/sqrt(d) by default. workspace:
    device memory of cache_attention_workspace_size bytes, by default allocated here; one call at a
    time may use it."""
    step = _step_desc(cache, q, q.shape[1], page_table, kv_lens, cu_new, status)
    c = cache.desc
    _check(window is None or window >= 1, "window must be at least 1")
    _check(sinks >= 0, "sinks must not be negative")
    _check(out is None or (out.shape == q.shape and out.dtype == q.dtype), "out must be like q")
    tq, to = _view3(q), None if out is None else _view3(out)
    dev = _one_device(q, cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale, page_table, kv_lens, cu_new, out,
                      workspace, status)
    lib = load_library()

    def body(raw):
        o = torch.empty_like(q) if out is None else out
        if step.T == 0:
            if status is not None:
                status.zero_()
            return o
        if workspace is None:
            n = lib.sla2_cache_attention_workspace_size(c, step)
            ws = q.new_empty(max(n, 1), dtype=torch.uint8)
        else:
            ws = workspace
        r = lib.sla2_cache_attention(c, step, tq, _view3(o) if to is None else to, 0x7fffffff if window is None else min(window, 0x7fffffff),
                                     min(sinks, 0x7fffffff), c.d ** -0.5 if scale is None else scale,
                                     ws.data_ptr(), ws.numel() * ws.element_size(), raw)
        if r != 0:
            raise Sla2Error(r, "sla2_cache_attention")
        return o

    return _enqueue(dev, stream, (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale, q, page_table, kv_lens,
                                  cu_new, out, workspace, status), body)

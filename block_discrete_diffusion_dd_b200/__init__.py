"""Python binding of libdd, the B200 (sm_100a) library for one denoising step
of block discrete-diffusion decoding ("DiffusionGemma Technical Report",
paperfeed review, "The mechanism: an AR model turned inside out").

This module only marshals arguments: torch tensors in, raw device pointers
and sizes out to the C ABI (include/dd.h); torch provides device memory and
streams.  Every step of the computation runs in the library's CUDA kernels.
There is no CPU fallback: if libdd.so is missing or the GPU is unusable,
calls raise.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdd.so")

DD_BF16, DD_F32, DD_E4M3 = 0, 1, 2
STATUS = {0: "DD_OK", 1: "DD_ERR_INVALID_ARG", 2: "DD_ERR_UNSUPPORTED", 3: "DD_ERR_WORKSPACE",
          4: "DD_ERR_CUDA", 5: "DD_ERR_DEVICE_TIMEOUT", 6: "DD_ERR_DEVICE_BOUNDS"}

# every symbol include/dd.h declares
EXPORTS = (
    "dd_canvas_attn_workspace", "dd_canvas_attn", "dd_sample_renoise_workspace",
    "dd_sample_renoise", "dd_init_canvas", "dd_denoise_block_workspace", "dd_denoise_block",
    "dd_workspace_init", "dd_query_device_error", "dd_status_string", "dd_last_error",
    "dd_launch_count", "dd_reset_launch_count", "dd_sample_renoise_noalloc",
    "dd_entropy_accept", "dd_stop_check", "dd_denoise_block_adaptive_workspace",
    "dd_denoise_block_adaptive", "dd_canvas_attn_fp8", "dd_denoise_block_graph_create",
    "dd_denoise_block_graph_launch", "dd_denoise_block_graph_destroy",
    "dd_soft_embed_workspace", "dd_soft_embed", "dd_denoise_block_fp8",
    "dd_denoise_block_adaptive_graph_create", "dd_denoise_block_adaptive_graph_launch",
    "dd_denoise_block_adaptive_graph_destroy", "dd_ffw_workspace", "dd_ffw",
    "dd_self_condition_workspace", "dd_self_condition", "dd_set_test_stall_ns",
    "dd_cache_workspace", "dd_cache_append", "dd_cache_read", "dd_paged_attn_workspace",
    "dd_paged_attn", "dd_verify_draft_workspace", "dd_verify_draft",
)


class DDError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{STATUS.get(status, status)}: {detail}")
        self.status = status


class AttnDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("canvas", ctypes.c_int), ("heads_q", ctypes.c_int),
                ("heads_kv", ctypes.c_int), ("head_dim", ctypes.c_int), ("scale", ctypes.c_float),
                ("dtype", ctypes.c_int)]


class Fp8Scales(ctypes.Structure):
    _fields_ = [("q", ctypes.c_float), ("k", ctypes.c_float), ("v", ctypes.c_float)]


class SampleParams(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("renoise_rate", ctypes.c_float),
                ("seed", ctypes.c_uint64), ("step", ctypes.c_uint32),
                ("row_offset", ctypes.c_uint32)]


class _PagedCacheC(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("heads_kv", ctypes.c_int), ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


class _PagedBatchC(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("max_pages", ctypes.c_int), ("total_new", ctypes.c_int),
                ("max_new", ctypes.c_int), ("page_table", ctypes.c_void_p),
                ("cu_new", ctypes.c_void_p), ("kv_len", ctypes.c_void_p)]


class VerifyParams(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("draft_temperature", ctypes.c_float)]


_lib = None


def load() -> ctypes.CDLL:
    """Load libdd.so (built in-tree by build.build()); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libdd.so not found at {LIB_PATH}: run "
                           "block_discrete_diffusion_dd_b200.build.build() first")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, u32, u64, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint32,
                                 ctypes.c_uint64, ctypes.c_size_t)
    f32 = ctypes.c_float
    D = ctypes.POINTER(AttnDesc)
    lib.dd_canvas_attn_workspace.restype = sz
    lib.dd_canvas_attn_workspace.argtypes = [D, P]
    lib.dd_canvas_attn.restype = i32
    lib.dd_canvas_attn.argtypes = [D, P, P, P, P, P, P, P, P, P, P, sz, P]
    lib.dd_canvas_attn_fp8.restype = i32
    lib.dd_canvas_attn_fp8.argtypes = [D, P, P, P, P, P, P, P, ctypes.POINTER(Fp8Scales), P, P, P,
                                       sz, P]
    lib.dd_sample_renoise_workspace.restype = sz
    lib.dd_sample_renoise_workspace.argtypes = [i32, i32, i32]
    lib.dd_sample_renoise.restype = i32
    lib.dd_sample_renoise.argtypes = [P, i32, i32, i32, i64, ctypes.POINTER(SampleParams), P, P, P,
                                      P, P, P, sz, P]
    lib.dd_sample_renoise_noalloc.restype = i32
    lib.dd_sample_renoise_noalloc.argtypes = [P, i32, i32, i32, i64, ctypes.POINTER(SampleParams),
                                              P, P, P, P, P, P]
    lib.dd_init_canvas.restype = i32
    lib.dd_init_canvas.argtypes = [P, i32, i32, u64, u32, P]
    lib.dd_denoise_block_workspace.restype = sz
    lib.dd_denoise_block_workspace.argtypes = [D, P, i32]
    lib.dd_denoise_block.restype = i32
    lib.dd_denoise_block.argtypes = [D, i32, P, P, P, P, P, P, P, P, P, i32, P, P, u64, u32, P, P,
                                     P, P, sz, P]
    lib.dd_denoise_block_fp8.restype = i32
    lib.dd_denoise_block_fp8.argtypes = [D, i32, P, P, P, P, P, P, P, P, P, P, i32, P, P, u64, u32,
                                         P, P, P, P, sz, P]
    lib.dd_denoise_block_graph_create.restype = i32
    lib.dd_denoise_block_graph_create.argtypes = [ctypes.POINTER(P), D, i32, P, P, P, P, P, P, P,
                                                  P, P, i32, P, P, u64, u32, P, P, P, P, sz]
    lib.dd_denoise_block_graph_launch.restype = i32
    lib.dd_denoise_block_graph_launch.argtypes = [P, P]
    lib.dd_denoise_block_graph_destroy.restype = i32
    lib.dd_denoise_block_graph_destroy.argtypes = [P]
    lib.dd_denoise_block_adaptive_graph_create.restype = i32
    lib.dd_denoise_block_adaptive_graph_create.argtypes = [ctypes.POINTER(P), D, i32, P, P, P, P,
                                                           P, P, P, P, P, i32, P, f32, f32, u64,
                                                           u32, P, P, P, P, P, sz]
    lib.dd_denoise_block_adaptive_graph_launch.restype = i32
    lib.dd_denoise_block_adaptive_graph_launch.argtypes = [P, P]
    lib.dd_denoise_block_adaptive_graph_destroy.restype = i32
    lib.dd_denoise_block_adaptive_graph_destroy.argtypes = [P]
    lib.dd_soft_embed_workspace.restype = sz
    lib.dd_soft_embed_workspace.argtypes = [i32, i32, i32]
    lib.dd_soft_embed.restype = i32
    lib.dd_soft_embed.argtypes = [P, i32, i32, i32, i64, ctypes.c_float, P, i32, P, P, sz, P]
    lib.dd_set_test_stall_ns.restype = None
    lib.dd_set_test_stall_ns.argtypes = [u64]
    lib.dd_ffw_workspace.restype = sz
    lib.dd_ffw_workspace.argtypes = [i32, i32, i32]
    lib.dd_ffw.restype = i32
    lib.dd_ffw.argtypes = [P, i32, i32, i32, P, P, P, P, P, P, sz, P]
    lib.dd_self_condition_workspace.restype = sz
    lib.dd_self_condition_workspace.argtypes = [i32, i32, i32, i32]
    lib.dd_self_condition.restype = i32
    lib.dd_self_condition.argtypes = [P, i32, i32, i32, i64, ctypes.c_float, P, i32, P, P, i32, P,
                                      P, P, P, P, sz, P]
    lib.dd_entropy_accept.restype = i32
    lib.dd_entropy_accept.argtypes = [P, P, i32, i32, i32, f32, u64, u32, u32, P, P, P]
    lib.dd_stop_check.restype = i32
    lib.dd_stop_check.argtypes = [P, P, P, i32, i32, f32, ctypes.c_int32, P, P, P]
    lib.dd_denoise_block_adaptive_workspace.restype = sz
    lib.dd_denoise_block_adaptive_workspace.argtypes = [D, P, i32]
    lib.dd_denoise_block_adaptive.restype = i32
    lib.dd_denoise_block_adaptive.argtypes = [D, i32, P, P, P, P, P, P, P, P, P, i32, P, f32, f32,
                                              u64, u32, P, P, P, ctypes.POINTER(ctypes.c_int),
                                              P, sz, P]
    PC, PB = ctypes.POINTER(_PagedCacheC), ctypes.POINTER(_PagedBatchC)
    lib.dd_cache_workspace.restype = sz
    lib.dd_cache_workspace.argtypes = []
    lib.dd_cache_append.restype = i32
    lib.dd_cache_append.argtypes = [PC, PB, P, i64, P, i64, P, sz, P]
    lib.dd_cache_read.restype = i32
    lib.dd_cache_read.argtypes = [PC, i32, i32, P, P, i32, P, P, P, sz, P]
    lib.dd_paged_attn_workspace.restype = sz
    lib.dd_paged_attn_workspace.argtypes = [PC, PB, i32]
    lib.dd_paged_attn.restype = i32
    lib.dd_paged_attn.argtypes = [PC, PB, i32, P, i64, f32, i32, P, P, P, sz, P]
    lib.dd_verify_draft_workspace.restype = sz
    lib.dd_verify_draft_workspace.argtypes = [i32, i32, i32]
    lib.dd_verify_draft.restype = i32
    lib.dd_verify_draft.argtypes = [ctypes.POINTER(VerifyParams), i32, i32, i32, i32, P, i64, P,
                                    i64, P, P, P, P, P, P, P, P, P, sz, P]
    lib.dd_workspace_init.restype = i32
    lib.dd_workspace_init.argtypes = [P, sz, P]
    lib.dd_query_device_error.restype = i32
    lib.dd_query_device_error.argtypes = [P, P]
    lib.dd_status_string.restype = ctypes.c_char_p
    lib.dd_status_string.argtypes = [i32]
    lib.dd_last_error.restype = ctypes.c_char_p
    lib.dd_last_error.argtypes = []
    lib.dd_launch_count.restype = u64
    lib.dd_launch_count.argtypes = []
    lib.dd_reset_launch_count.restype = None
    lib.dd_reset_launch_count.argtypes = []
    _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        raise DDError(status, load().dd_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream: Optional[torch.cuda.Stream]):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return DD_BF16
    if t.dtype == torch.float32:
        return DD_F32
    if t.dtype == torch.float8_e4m3fn:
        return DD_E4M3
    raise TypeError(f"unsupported dtype {t.dtype} (bf16, fp32 or float8_e4m3fn)")


def _host_i32(x) -> np.ndarray:
    if isinstance(x, torch.Tensor):
        x = x.cpu().numpy()
    return np.ascontiguousarray(np.asarray(x, dtype=np.int32))


def new_workspace(nbytes: int, device=None, stream=None) -> torch.Tensor:
    """A device workspace (torch-owned) with its error word cleared."""
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    ws = torch.empty(max(int(nbytes), 256) + 256, dtype=torch.uint8, device=dev)
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + max(int(nbytes), 256)]
    _check(load().dd_workspace_init(_ptr(ws), ws.numel(), _stream(stream)))
    return ws


def attn_desc(q: torch.Tensor, kc: torch.Tensor, scale: Optional[float] = None) -> AttnDesc:
    B, C, Hq, D = q.shape
    Hkv = kc.shape[2]
    return AttnDesc(B, C, Hq, Hkv, D, float(scale if scale is not None else D ** -0.5),
                    _dtype_code(q))


def canvas_attn_workspace_bytes(desc: AttnDesc, cu_prefix_host) -> int:
    cu = _host_i32(cu_prefix_host)
    return int(load().dd_canvas_attn_workspace(ctypes.byref(desc), cu.ctypes.data_as(ctypes.c_void_p)))


def canvas_attn(q, kc, vc, kp, vp, cu_prefix, cu_prefix_host=None, scale=None, out=None,
                lse=None, want_lse=False, workspace=None, stream=None):
    """dd_canvas_attn: q [B,C,Hq,D], kc/vc [B,C,Hkv,D], kp/vp [sumL,Hkv,D],
    cu_prefix int32 [B+1] on the device.  Returns (out, lse or None)."""
    lib = load()
    desc = attn_desc(q, kc, scale)
    cu_h = _host_i32(cu_prefix if cu_prefix_host is None else cu_prefix_host)
    if out is None:
        out = torch.empty_like(q)
    if want_lse and lse is None:
        lse = torch.empty((desc.batch, desc.heads_q, desc.canvas), dtype=torch.float32,
                          device=q.device)
    if workspace is None:
        workspace = new_workspace(canvas_attn_workspace_bytes(desc, cu_h), q.device, stream)
    _check(lib.dd_canvas_attn(ctypes.byref(desc), _ptr(q), _ptr(kc), _ptr(vc), _ptr(kp), _ptr(vp),
                              _ptr(cu_prefix), cu_h.ctypes.data_as(ctypes.c_void_p), _ptr(out),
                              _ptr(lse), _ptr(workspace), workspace.numel(), _stream(stream)))
    return out, lse


def canvas_attn_fp8(q, kc, vc, kp, vp, cu_prefix, scales, cu_prefix_host=None, scale=None,
                    out=None, lse=None, want_lse=False, workspace=None, stream=None):
    """dd_canvas_attn_fp8: float8_e4m3fn q [B,C,Hq,D], kc/vc [B,C,Hkv,D],
    kp/vp [sumL,Hkv,D]; scales = (f_q, f_k, f_v) per-tensor factors.
    Returns (out bf16 [B,C,Hq,D], lse or None)."""
    lib = load()
    desc = attn_desc(q, kc, scale)
    cu_h = _host_i32(cu_prefix if cu_prefix_host is None else cu_prefix_host)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    if want_lse and lse is None:
        lse = torch.empty((desc.batch, desc.heads_q, desc.canvas), dtype=torch.float32,
                          device=q.device)
    if workspace is None:
        workspace = new_workspace(canvas_attn_workspace_bytes(desc, cu_h), q.device, stream)
    f = Fp8Scales(*(float(x) for x in scales))
    _check(lib.dd_canvas_attn_fp8(ctypes.byref(desc), _ptr(q), _ptr(kc), _ptr(vc), _ptr(kp),
                                  _ptr(vp), _ptr(cu_prefix), cu_h.ctypes.data_as(ctypes.c_void_p),
                                  ctypes.byref(f), _ptr(out), _ptr(lse), _ptr(workspace),
                                  workspace.numel(), _stream(stream)))
    return out, lse


def sample_workspace_bytes(rows: int, vocab: int, dtype=torch.bfloat16) -> int:
    code = DD_BF16 if dtype == torch.bfloat16 else DD_F32
    return int(load().dd_sample_renoise_workspace(rows, vocab, code))


def sample_renoise(logits: torch.Tensor, temperature: float, rate: float, seed: int, step: int,
                   row_offset: int = 0, rows: Optional[int] = None, vocab: Optional[int] = None,
                   row_stride: Optional[int] = None, outputs: Optional[dict] = None,
                   workspace=None, stream=None) -> dict:
    """dd_sample_renoise over logits [R, V] (bf16/fp32).  Returns a dict of
    device tensors: tokens, pred, conf, entropy, renoised."""
    lib = load()
    R = logits.shape[0] if rows is None else rows
    V = logits.shape[-1] if vocab is None else vocab
    stride = logits.stride(0) if row_stride is None else row_stride
    dev = logits.device
    o = outputs if outputs is not None else {
        "tokens": torch.empty(R, dtype=torch.int32, device=dev),
        "pred": torch.empty(R, dtype=torch.int32, device=dev),
        "conf": torch.empty(R, dtype=torch.float32, device=dev),
        "entropy": torch.empty(R, dtype=torch.float32, device=dev),
        "renoised": torch.empty(R, dtype=torch.uint8, device=dev),
    }
    if workspace is None:
        workspace = new_workspace(sample_workspace_bytes(R, V, logits.dtype), dev, stream)
    prm = SampleParams(float(temperature), float(rate), int(seed), int(step), int(row_offset))
    _check(lib.dd_sample_renoise(_ptr(logits), _dtype_code(logits), R, V, stride,
                                 ctypes.byref(prm), _ptr(o["tokens"]), _ptr(o.get("pred")),
                                 _ptr(o["conf"]), _ptr(o.get("entropy")), _ptr(o.get("renoised")),
                                 _ptr(workspace), workspace.numel(), _stream(stream)))
    return o


def sample_renoise_noalloc(logits: torch.Tensor, temperature: float, rate: float, seed: int,
                           step: int, row_offset: int = 0, outputs: Optional[dict] = None,
                           stream=None) -> dict:
    """dd_sample_renoise_noalloc: the sampler step with the library's static
    scratch instead of a workspace (for callers that must not allocate).
    Calls must not overlap on the GPU; see include/dd.h."""
    lib = load()
    R, V = logits.shape[0], logits.shape[-1]
    dev = logits.device
    o = outputs if outputs is not None else {
        "tokens": torch.empty(R, dtype=torch.int32, device=dev),
        "pred": torch.empty(R, dtype=torch.int32, device=dev),
        "conf": torch.empty(R, dtype=torch.float32, device=dev),
        "entropy": torch.empty(R, dtype=torch.float32, device=dev),
        "renoised": torch.empty(R, dtype=torch.uint8, device=dev),
    }
    prm = SampleParams(float(temperature), float(rate), int(seed), int(step), int(row_offset))
    _check(lib.dd_sample_renoise_noalloc(_ptr(logits), _dtype_code(logits), R, V,
                                         logits.stride(0), ctypes.byref(prm), _ptr(o["tokens"]),
                                         _ptr(o.get("pred")), _ptr(o["conf"]),
                                         _ptr(o.get("entropy")), _ptr(o.get("renoised")),
                                         _stream(stream)))
    return o


def init_canvas(rows: int, vocab: int, seed: int, row_offset: int = 0, out=None, device=None,
                stream=None) -> torch.Tensor:
    if out is None:
        out = torch.empty(rows, dtype=torch.int32, device=device or "cuda")
    _check(load().dd_init_canvas(_ptr(out), rows, vocab, int(seed), int(row_offset),
                                 _stream(stream)))
    return out


def denoise_block_workspace_bytes(desc: AttnDesc, cu_prefix_host, vocab: int) -> int:
    cu = _host_i32(cu_prefix_host)
    return int(load().dd_denoise_block_workspace(ctypes.byref(desc),
                                                 cu.ctypes.data_as(ctypes.c_void_p), vocab))


def denoise_block(q_steps, kc_steps, vc_steps, kp, vp, cu_prefix, logits_steps,
                  rates: Sequence[float], temperatures: Sequence[float], seed: int, step0: int = 0,
                  cu_prefix_host=None, scale=None, attn_out=None, canvas=None,
                  canvas_history=None, conf_steps=None, keep_history=True, workspace=None,
                  stream=None) -> dict:
    """dd_denoise_block: S steps of attention + sampler/re-noise.

    q_steps [S,B,C,Hq,D], kc/vc_steps [S,B,C,Hkv,D], logits_steps [S,B*C,V].
    Returns dict(attn_out, canvas, canvas_history, conf_steps)."""
    return _block_loop(None, q_steps, kc_steps, vc_steps, kp, vp, cu_prefix, logits_steps, rates,
                       temperatures, seed, step0, cu_prefix_host, scale, attn_out, canvas,
                       canvas_history, conf_steps, keep_history, workspace, stream)


def denoise_block_fp8(q_steps, kc_steps, vc_steps, kp, vp, cu_prefix, scales_steps,
                      logits_steps, rates: Sequence[float], temperatures: Sequence[float],
                      seed: int, step0: int = 0, cu_prefix_host=None, scale=None, attn_out=None,
                      canvas=None, canvas_history=None, conf_steps=None, keep_history=True,
                      workspace=None, stream=None) -> dict:
    """dd_denoise_block_fp8: as denoise_block with float8_e4m3fn attention
    inputs, scales_steps = one (f_q, f_k, f_v) per step, bf16 logits; the
    attention output is bf16."""
    return _block_loop(scales_steps, q_steps, kc_steps, vc_steps, kp, vp, cu_prefix, logits_steps,
                       rates, temperatures, seed, step0, cu_prefix_host, scale, attn_out, canvas,
                       canvas_history, conf_steps, keep_history, workspace, stream)


def _block_loop(scales_steps, q_steps, kc_steps, vc_steps, kp, vp, cu_prefix, logits_steps, rates,
                temperatures, seed, step0, cu_prefix_host, scale, attn_out, canvas,
                canvas_history, conf_steps, keep_history, workspace, stream) -> dict:
    lib = load()
    S = q_steps.shape[0]
    desc = attn_desc(q_steps[0], kc_steps[0], scale)
    cu_h = _host_i32(cu_prefix if cu_prefix_host is None else cu_prefix_host)
    V = logits_steps.shape[-1]
    R = desc.batch * desc.canvas
    dev = q_steps.device
    if attn_out is None:
        attn_out = torch.empty(q_steps.shape, device=dev, dtype=(
            q_steps.dtype if scales_steps is None else torch.bfloat16))
    if canvas is None:
        canvas = torch.empty(R, dtype=torch.int32, device=dev)
    if keep_history and canvas_history is None:
        canvas_history = torch.empty((S, R), dtype=torch.int32, device=dev)
    if keep_history and conf_steps is None:
        conf_steps = torch.empty((S, R), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = new_workspace(denoise_block_workspace_bytes(desc, cu_h, V), dev, stream)
    rates_h = np.ascontiguousarray(np.asarray(rates, dtype=np.float32))
    temps_h = np.ascontiguousarray(np.asarray(temperatures, dtype=np.float32))
    assert rates_h.size >= S and temps_h.size >= S
    head = (ctypes.byref(desc), S, _ptr(q_steps), _ptr(kc_steps), _ptr(vc_steps), _ptr(kp),
            _ptr(vp), _ptr(cu_prefix), cu_h.ctypes.data_as(ctypes.c_void_p))
    tail = (_ptr(attn_out), _ptr(logits_steps), V, rates_h.ctypes.data_as(ctypes.c_void_p),
            temps_h.ctypes.data_as(ctypes.c_void_p), int(seed), int(step0), _ptr(canvas),
            _ptr(canvas_history), _ptr(conf_steps), _ptr(workspace), workspace.numel(),
            _stream(stream))
    if scales_steps is None:
        _check(lib.dd_denoise_block(*head, *tail))
    else:
        assert len(scales_steps) >= S
        f = (Fp8Scales * max(S, 1))(*(Fp8Scales(*(float(x) for x in scales_steps[i]))
                                      for i in range(S)))
        _check(lib.dd_denoise_block_fp8(*head, ctypes.cast(f, ctypes.c_void_p), *tail))
    return {"attn_out": attn_out, "canvas": canvas, "canvas_history": canvas_history,
            "conf_steps": conf_steps}


def soft_embed_workspace_bytes(rows: int, vocab: int, d: int) -> int:
    return int(load().dd_soft_embed_workspace(rows, vocab, d))


def soft_embed(logits: torch.Tensor, temperature: float, emb: torch.Tensor, out=None,
               rows: Optional[int] = None, vocab: Optional[int] = None,
               row_stride: Optional[int] = None, workspace=None, stream=None) -> torch.Tensor:
    """dd_soft_embed: softmax(logits / temperature) @ emb, bf16 [rows, d]."""
    lib = load()
    R = logits.shape[0] if rows is None else rows
    V = logits.shape[-1] if vocab is None else vocab
    stride = logits.stride(0) if row_stride is None else row_stride
    d = emb.shape[-1]
    if out is None:
        out = torch.empty((R, d), dtype=torch.bfloat16, device=logits.device)
    if workspace is None:
        workspace = new_workspace(soft_embed_workspace_bytes(R, V, d), logits.device, stream)
    _check(lib.dd_soft_embed(_ptr(logits), _dtype_code(logits), R, V, stride, float(temperature),
                             _ptr(emb), d, _ptr(out), _ptr(workspace), workspace.numel(),
                             _stream(stream)))
    return out


def ffw(u: torch.Tensor, w1: torch.Tensor, b1: torch.Tensor, w2: torch.Tensor,
        b2: torch.Tensor, out=None, workspace=None, stream=None) -> torch.Tensor:
    """dd_ffw: the self-conditioning MLP GELU(u w1 + b1) w2 + b2, bf16
    [rows, d] (u [rows, d], w1 [d, h], b1 [h], w2 [h, d], b2 [d], bf16)."""
    lib = load()
    R, d = u.shape
    h = w1.shape[1]
    if out is None:
        out = torch.empty((R, d), dtype=torch.bfloat16, device=u.device)
    if workspace is None:
        workspace = new_workspace(int(lib.dd_ffw_workspace(R, d, h)), u.device, stream)
    _check(lib.dd_ffw(_ptr(u), R, d, h, _ptr(w1), _ptr(b1), _ptr(w2), _ptr(b2), _ptr(out),
                      _ptr(workspace), workspace.numel(), _stream(stream)))
    return out


def self_condition(logits: torch.Tensor, temperature: float, emb: torch.Tensor,
                   w1: torch.Tensor, b1: torch.Tensor, w2: torch.Tensor, b2: torch.Tensor,
                   out=None, u_out=None, workspace=None, stream=None) -> torch.Tensor:
    """dd_self_condition: z = FFW(softmax(logits / temperature) emb), bf16
    [rows, d]; u_out (optional, bf16 [rows, d]) receives the soft embedding."""
    lib = load()
    R, V = logits.shape
    d = emb.shape[1]
    h = w1.shape[1]
    if out is None:
        out = torch.empty((R, d), dtype=torch.bfloat16, device=logits.device)
    if workspace is None:
        workspace = new_workspace(int(lib.dd_self_condition_workspace(R, V, d, h)),
                                  logits.device, stream)
    _check(lib.dd_self_condition(_ptr(logits), _dtype_code(logits), R, V, logits.stride(0),
                                 float(temperature), _ptr(emb), d, _ptr(w1), _ptr(b1), h,
                                 _ptr(w2), _ptr(b2), _ptr(out), _ptr(u_out), _ptr(workspace),
                                 workspace.numel(), _stream(stream)))
    return out


class BlockGraph:
    """dd_denoise_block captured once (dd_denoise_block_graph_create) and
    replayed with one launch (launch()).  Holds every captured tensor, so the
    buffers outlive the graph; new inputs enter by writing into them
    (`tensors` maps the argument names to those tensors)."""

    _prefix = "dd_denoise_block_graph"

    def __init__(self, handle, tensors: dict, keep: tuple):
        self._h = handle
        self.tensors = tensors
        self._keep = keep

    def launch(self, stream=None):
        if self._h is None:
            raise RuntimeError(f"{type(self).__name__}: destroyed")
        _check(getattr(load(), self._prefix + "_launch")(self._h, _stream(stream)))
        return self.tensors

    def destroy(self):
        if self._h is not None:
            h, self._h = self._h, None
            _check(getattr(load(), self._prefix + "_destroy")(h))

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def denoise_block_graph(q_steps, kc_steps, vc_steps, kp, vp, cu_prefix, logits_steps,
                        rates: Sequence[float], temperatures: Sequence[float], seed: int,
                        step0: int = 0, cu_prefix_host=None, scale=None, attn_out=None,
                        canvas=None, canvas_history=None, conf_steps=None, keep_history=True,
                        workspace=None) -> BlockGraph:
    """dd_denoise_block_graph_create with the arguments of denoise_block."""
    lib = load()
    S = q_steps.shape[0]
    desc = attn_desc(q_steps[0], kc_steps[0], scale)
    cu_h = _host_i32(cu_prefix if cu_prefix_host is None else cu_prefix_host)
    V = logits_steps.shape[-1]
    R = desc.batch * desc.canvas
    dev = q_steps.device
    if attn_out is None:
        attn_out = torch.empty_like(q_steps)
    if canvas is None:
        canvas = torch.empty(R, dtype=torch.int32, device=dev)
    if keep_history and canvas_history is None:
        canvas_history = torch.empty((S, R), dtype=torch.int32, device=dev)
    if keep_history and conf_steps is None:
        conf_steps = torch.empty((S, R), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = new_workspace(denoise_block_workspace_bytes(desc, cu_h, V), dev)
    rates_h = np.ascontiguousarray(np.asarray(rates, dtype=np.float32))
    temps_h = np.ascontiguousarray(np.asarray(temperatures, dtype=np.float32))
    assert rates_h.size >= S and temps_h.size >= S
    h = ctypes.c_void_p()
    _check(lib.dd_denoise_block_graph_create(
        ctypes.byref(h), ctypes.byref(desc), S, _ptr(q_steps), _ptr(kc_steps), _ptr(vc_steps),
        _ptr(kp), _ptr(vp), _ptr(cu_prefix), cu_h.ctypes.data_as(ctypes.c_void_p),
        _ptr(attn_out), _ptr(logits_steps), V, rates_h.ctypes.data_as(ctypes.c_void_p),
        temps_h.ctypes.data_as(ctypes.c_void_p), int(seed), int(step0), _ptr(canvas),
        _ptr(canvas_history), _ptr(conf_steps), _ptr(workspace), workspace.numel()))
    tensors = {"q_steps": q_steps, "kc_steps": kc_steps, "vc_steps": vc_steps, "kp": kp, "vp": vp,
               "cu_prefix": cu_prefix, "logits_steps": logits_steps, "attn_out": attn_out,
               "canvas": canvas, "canvas_history": canvas_history, "conf_steps": conf_steps,
               "workspace": workspace}
    return BlockGraph(h, tensors, (cu_h, rates_h, temps_h))


def entropy_accept(entropy: torch.Tensor, pred: torch.Tensor, canvas: int, budget: float,
                   seed: int, step: int, vocab: int, row_offset: int = 0, tokens=None,
                   accepted=None, stream=None) -> dict:
    """dd_entropy_accept: the pages' entropy-budget acceptance per canvas."""
    R = entropy.numel()
    if tokens is None:
        tokens = torch.empty(R, dtype=torch.int32, device=entropy.device)
    if accepted is None:
        accepted = torch.empty(R, dtype=torch.uint8, device=entropy.device)
    _check(load().dd_entropy_accept(_ptr(entropy), _ptr(pred), R // canvas, canvas, vocab,
                                    float(budget), int(seed), int(step), int(row_offset),
                                    _ptr(tokens), _ptr(accepted), _stream(stream)))
    return {"tokens": tokens, "accepted": accepted}


def stop_check(entropy: torch.Tensor, pred: torch.Tensor, pred_prev, canvas: int,
               threshold: float, step: int, done: torch.Tensor, halt_step: torch.Tensor,
               stream=None):
    """dd_stop_check: updates done [B] and halt_step [B] in place."""
    _check(load().dd_stop_check(_ptr(entropy), _ptr(pred), _ptr(pred_prev),
                                entropy.numel() // canvas, canvas, float(threshold), int(step),
                                _ptr(done), _ptr(halt_step), _stream(stream)))


def denoise_block_adaptive(q_steps, kc_steps, vc_steps, kp, vp, cu_prefix, logits_steps,
                           temperatures: Sequence[float], budget: float, stop_entropy: float,
                           seed: int, step0: int = 0, cu_prefix_host=None, scale=None,
                           attn_out=None, canvas=None, keep_history=True, workspace=None,
                           stream=None) -> dict:
    """dd_denoise_block_adaptive: the block loop under the pages' policy.

    Returns dict(canvas, canvas_history [steps_run, R] or None, halt_step [B],
    steps_run)."""
    lib = load()
    S = q_steps.shape[0]
    desc = attn_desc(q_steps[0], kc_steps[0], scale)
    cu_h = _host_i32(cu_prefix if cu_prefix_host is None else cu_prefix_host)
    V = logits_steps.shape[-1]
    R = desc.batch * desc.canvas
    dev = q_steps.device
    if attn_out is None:
        attn_out = torch.empty_like(q_steps)
    if canvas is None:
        canvas = torch.zeros(R, dtype=torch.int32, device=dev)
    history = torch.empty((S, R), dtype=torch.int32, device=dev) if keep_history else None
    halt = torch.empty(desc.batch, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = new_workspace(int(lib.dd_denoise_block_adaptive_workspace(
            ctypes.byref(desc), cu_h.ctypes.data_as(ctypes.c_void_p), V)), dev, stream)
    temps_h = np.ascontiguousarray(np.asarray(temperatures, dtype=np.float32))
    assert temps_h.size >= S
    steps_run = ctypes.c_int(0)
    _check(lib.dd_denoise_block_adaptive(
        ctypes.byref(desc), S, _ptr(q_steps), _ptr(kc_steps), _ptr(vc_steps), _ptr(kp), _ptr(vp),
        _ptr(cu_prefix), cu_h.ctypes.data_as(ctypes.c_void_p), _ptr(attn_out),
        _ptr(logits_steps), V, temps_h.ctypes.data_as(ctypes.c_void_p), float(budget),
        float(stop_entropy), int(seed), int(step0), _ptr(canvas), _ptr(history), _ptr(halt),
        ctypes.byref(steps_run), _ptr(workspace), workspace.numel(), _stream(stream)))
    n = steps_run.value
    return {"canvas": canvas, "canvas_history": None if history is None else history[:n],
            "halt_step": halt, "steps_run": n}


class AdaptiveGraph(BlockGraph):
    """dd_denoise_block_adaptive captured once with the loop on the device
    (dd_denoise_block_adaptive_graph_create); launch() replays it without
    any host synchronisation.  tensors["steps_run"] is a device int32 [1]."""
    _prefix = "dd_denoise_block_adaptive_graph"


def denoise_block_adaptive_graph(q_steps, kc_steps, vc_steps, kp, vp, cu_prefix, logits_steps,
                                 temperatures: Sequence[float], budget: float,
                                 stop_entropy: float, seed: int, step0: int = 0,
                                 cu_prefix_host=None, scale=None, attn_out=None, canvas=None,
                                 keep_history=True, workspace=None) -> AdaptiveGraph:
    """dd_denoise_block_adaptive_graph_create with the arguments of
    denoise_block_adaptive."""
    lib = load()
    S = q_steps.shape[0]
    desc = attn_desc(q_steps[0], kc_steps[0], scale)
    cu_h = _host_i32(cu_prefix if cu_prefix_host is None else cu_prefix_host)
    V = logits_steps.shape[-1]
    R = desc.batch * desc.canvas
    dev = q_steps.device
    if attn_out is None:
        attn_out = torch.empty_like(q_steps)
    if canvas is None:
        canvas = torch.zeros(R, dtype=torch.int32, device=dev)
    history = torch.empty((S, R), dtype=torch.int32, device=dev) if keep_history else None
    halt = torch.empty(desc.batch, dtype=torch.int32, device=dev)
    steps_run = torch.zeros(1, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = new_workspace(int(lib.dd_denoise_block_adaptive_workspace(
            ctypes.byref(desc), cu_h.ctypes.data_as(ctypes.c_void_p), V)), dev)
    temps_h = np.ascontiguousarray(np.asarray(temperatures, dtype=np.float32))
    assert temps_h.size >= S
    h = ctypes.c_void_p()
    _check(lib.dd_denoise_block_adaptive_graph_create(
        ctypes.byref(h), ctypes.byref(desc), S, _ptr(q_steps), _ptr(kc_steps), _ptr(vc_steps),
        _ptr(kp), _ptr(vp), _ptr(cu_prefix), cu_h.ctypes.data_as(ctypes.c_void_p),
        _ptr(attn_out), _ptr(logits_steps), V, temps_h.ctypes.data_as(ctypes.c_void_p),
        float(budget), float(stop_entropy), int(seed), int(step0), _ptr(canvas), _ptr(history),
        _ptr(halt), _ptr(steps_run), _ptr(workspace), workspace.numel()))
    tensors = {"q_steps": q_steps, "kc_steps": kc_steps, "vc_steps": vc_steps, "kp": kp, "vp": vp,
               "cu_prefix": cu_prefix, "logits_steps": logits_steps, "attn_out": attn_out,
               "canvas": canvas, "canvas_history": history, "halt_step": halt,
               "steps_run": steps_run, "workspace": workspace}
    return AdaptiveGraph(h, tensors, (cu_h, temps_h))


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


class _on:
    """Makes `device`, and `stream` if one is given, the current ones around a
    call, so that what the call allocates belongs to the stream that it runs
    on; `raw` is that stream's handle (a torch.cuda.Stream object costs more
    than a launch)."""
    __slots__ = ("raw", "_guard", "_caller")

    def __init__(self, device, stream):
        self._caller = None
        if stream is None:
            self._guard = (None if device.index == torch._C._cuda_getDevice()
                           else torch.cuda.device(device))
            self.raw = torch._C._cuda_getCurrentRawStream(device.index)
        else:
            _need(stream.device == device, f"a stream of {stream.device} for tensors on {device}")
            self._caller = torch.cuda.current_stream(device)
            self._guard = torch.cuda.stream(stream)
            self.raw = stream.cuda_stream

    def __enter__(self):
        if self._guard is not None:
            self._guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self._guard is not None:
            self._guard.__exit__(*exc)

    def lend(self, t: torch.Tensor) -> torch.Tensor:
        """A tensor allocated here and returned to a caller on another stream:
        its memory is not reused before that stream is done with it either."""
        if self._caller is not None:
            t.record_stream(self._caller)
        return t


def _own(workspace: torch.Tensor, device):
    if workspace.device != device or workspace.dtype != torch.uint8:
        raise ValueError(f"workspace: {workspace.dtype} on {workspace.device}, expected "
                         f"torch.uint8 on {device}")
    if not workspace.is_contiguous():  # (its size is counted by elements)
        raise ValueError("workspace must be contiguous")


def _packed(t: torch.Tensor, heads: int, dim: int, dtype, device, what: str) -> int:
    """Checks a packed [rows, heads, dim] tensor whose rows may lie apart (a
    view of a fused projection) and returns the elements between rows."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{what}: shape {tuple(shape)}, expected [rows, {heads}, {dim}]")
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{what}: {t.dtype} on {t.device}, expected {dtype} on {device}")
    s = t.stride()
    if (dim > 1 and s[2] != 1) or (heads > 1 and s[1] != dim):
        raise ValueError(f"{what}: a row's [heads, dim] must be contiguous")
    return s[0] if shape[0] > 1 else heads * dim


def _dense(t: torch.Tensor, shape, dtype, device, what: str):
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{what}: {t.dtype} on {t.device}, expected {dtype} on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


class PagedCache:
    """A paged K/V cache (dd_paged_cache): k, v [num_pages, heads_kv,
    page_size, head_dim] in bf16, or in float8_e4m3fn with uint8 k_scale,
    v_scale [num_pages, heads_kv, page_size] (byte s stands for 2^(s - 127)).
    The tensors stay the caller's; the object keeps them alive."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None):
        _need(k.is_cuda and k.numel() > 0, "k: a non-empty CUDA tensor is needed")
        _need(k.dim() == 4, f"k: shape {tuple(k.shape)}, expected [pages, heads, page_size, dim]")
        _dense(k, k.shape, k.dtype, k.device, "k")
        _dense(v, k.shape, k.dtype, k.device, "v")
        self.device, code = k.device, _dtype_code(k)
        if code == DD_E4M3:
            _need(k_scale is not None and v_scale is not None,
                  "an E4M3 cache needs k_scale and v_scale")
            for t, what in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                _dense(t, k.shape[:3], torch.uint8, k.device, what)
        else:
            _need(k_scale is None and v_scale is None, "only an E4M3 cache has scales")
        self._tensors = k, v, k_scale, v_scale
        self.num_pages, self.heads_kv, self.page_size, self.head_dim = k.shape

        def at(t):
            return None if t is None else t.data_ptr()

        self._c = _PagedCacheC(self.num_pages, self.page_size, self.heads_kv, self.head_dim, code,
                               at(k), at(v), at(k_scale), at(v_scale))
        self._ref = ctypes.byref(self._c)

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_scale = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])


def new_paged_cache(num_pages: int, page_size: int, heads_kv: int, head_dim: int,
                    dtype=torch.bfloat16, device="cuda") -> PagedCache:
    """An empty PagedCache of bf16 or float8_e4m3fn."""
    shape = (num_pages, heads_kv, page_size, head_dim)
    k, v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
    if dtype != torch.float8_e4m3fn:
        return PagedCache(k, v)
    return PagedCache(k, v, *(torch.full(shape[:3], 127, dtype=torch.uint8, device=device)
                              for _ in range(2)))


class PagedBatch:
    """The sequences of a call over a PagedCache (dd_paged_batch): page_table
    int32 [B, max_pages], cu_new int32 [B+1], kv_len int32 [B] (with the new
    tokens), all on the device; max_new bounds any sequence's new tokens.
    Their contents may change between calls; the tensors are kept alive."""

    def __init__(self, page_table: torch.Tensor, cu_new: torch.Tensor, kv_len: torch.Tensor,
                 max_new: int):
        self.max_new = max_new
        self._take(page_table, cu_new, kv_len)

    def _take(self, page_table, cu_new, kv_len):
        _need(page_table.dim() == 2, "page_table must be [batch, max_pages]")
        B, pages = page_table.shape
        _need(page_table.is_cuda, "page_table must be a CUDA tensor")
        dev = page_table.device
        _dense(page_table, (B, pages), torch.int32, dev, "page_table")
        _dense(cu_new, (B + 1,), torch.int32, dev, "cu_new")
        _dense(kv_len, (B,), torch.int32, dev, "kv_len")
        self.device, self.batch, self._tensors = dev, B, (page_table, cu_new, kv_len)
        self._struct = _PagedBatchC(B, pages, 0, 0, page_table.data_ptr(), cu_new.data_ptr(),
                                    kv_len.data_ptr())

    page_table = property(lambda self: self._tensors[0],
                          lambda self, t: self._take(t, self.cu_new, self.kv_len))
    cu_new = property(lambda self: self._tensors[1],
                      lambda self, t: self._take(self.page_table, t, self.kv_len))
    kv_len = property(lambda self: self._tensors[2],
                      lambda self, t: self._take(self.page_table, self.cu_new, t))

    def _c(self, total_new: int):
        c = self._struct
        if c.total_new != total_new or c.max_new != self.max_new:
            # a new one: a call on another host thread may be reading the last
            c = self._struct = _PagedBatchC(c.batch, c.max_pages, total_new, self.max_new,
                                            c.page_table, c.cu_new, c.kv_len)
        return c


def cache_append(cache: PagedCache, batch: PagedBatch, k_new: torch.Tensor, v_new: torch.Tensor,
                 workspace=None, stream=None):
    """dd_cache_append: writes bf16 k_new, v_new [total_new, heads_kv,
    head_dim] (rows may lie apart) at the batch's last positions."""
    lib, dev = load(), cache.device
    _need(batch.device == dev, "the batch and the cache are on different devices")
    ks = _packed(k_new, cache.heads_kv, cache.head_dim, torch.bfloat16, dev, "k_new")
    vs = _packed(v_new, cache.heads_kv, cache.head_dim, torch.bfloat16, dev, "v_new")
    _need(k_new.shape[0] == v_new.shape[0], "k_new and v_new have different numbers of rows")
    with _on(dev, stream) as on:
        if workspace is None:
            workspace = new_workspace(int(lib.dd_cache_workspace()), dev, stream)
        _own(workspace, dev)
        _check(lib.dd_cache_append(cache._ref, batch._c(k_new.shape[0]), k_new.data_ptr(), ks,
                                   v_new.data_ptr(), vs, workspace.data_ptr(), workspace.numel(),
                                   on.raw))


def cache_read(cache: PagedCache, page_table: torch.Tensor, cu_prefix: torch.Tensor,
               total: Optional[int] = None, k_out=None, v_out=None, workspace=None, stream=None):
    """dd_cache_read: the first cu_prefix[b+1] - cu_prefix[b] positions of
    every sequence, packed as canvas_attn takes them.  Returns (kp, vp), bf16
    [total, heads_kv, head_dim]; total defaults to k_out's rows."""
    lib, dev = load(), cache.device
    _need(page_table.dim() == 2, "page_table must be [batch, max_pages]")
    B, pages = page_table.shape
    _dense(page_table, (B, pages), torch.int32, dev, "page_table")
    _dense(cu_prefix, (B + 1,), torch.int32, dev, "cu_prefix")
    _need(total is not None or k_out is not None, "cache_read needs total or k_out")
    total = k_out.shape[0] if total is None else int(total)
    _need(total >= 0, f"total={total}")
    shape = (total, cache.heads_kv, cache.head_dim)
    with _on(dev, stream) as on:
        if k_out is None:
            k_out = on.lend(torch.empty(shape, dtype=torch.bfloat16, device=dev))
        if v_out is None:
            v_out = on.lend(torch.empty(shape, dtype=torch.bfloat16, device=dev))
        _dense(k_out, shape, torch.bfloat16, dev, "k_out")
        _dense(v_out, shape, torch.bfloat16, dev, "v_out")
        if workspace is None:
            workspace = new_workspace(int(lib.dd_cache_workspace()), dev, stream)
        _own(workspace, dev)
        _check(lib.dd_cache_read(cache._ref, B, pages, page_table.data_ptr(),
                                 cu_prefix.data_ptr(), total, k_out.data_ptr(), v_out.data_ptr(),
                                 workspace.data_ptr(), workspace.numel(), on.raw))
    return k_out, v_out


def paged_attn_workspace_bytes(cache: PagedCache, batch: PagedBatch, total_new: int,
                               heads_q: int) -> int:
    return int(load().dd_paged_attn_workspace(cache._ref, batch._c(total_new), heads_q))


def paged_attn(q: torch.Tensor, cache: PagedCache, batch: PagedBatch,
               scale: Optional[float] = None, causal: bool = True, out=None, lse=None,
               want_lse: bool = False, workspace=None, stream=None):
    """dd_paged_attn: attention of the batch's new tokens, q bf16 [total_new,
    heads_q, head_dim] (rows may lie apart), over the cache that holds their
    own K and V.  Returns (out [total_new, heads_q, head_dim], lse
    [total_new, heads_q] or None)."""
    lib, dev, D = load(), cache.device, cache.head_dim
    _need(q.dim() == 3, "q must be [total_new, heads_q, head_dim]")
    T, Hq = q.shape[0], q.shape[1]
    qs = _packed(q, Hq, D, torch.bfloat16, dev, "q")
    _need(batch.device == dev, "the batch and the cache are on different devices")
    with _on(dev, stream) as on:
        if out is None:
            out = on.lend(torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev))
        _dense(out, (T, Hq, D), torch.bfloat16, dev, "out")
        if want_lse and lse is None:
            lse = on.lend(torch.empty((T, Hq), dtype=torch.float32, device=dev))
        if lse is not None:
            _dense(lse, (T, Hq), torch.float32, dev, "lse")
        if workspace is None:
            workspace = new_workspace(paged_attn_workspace_bytes(cache, batch, T, Hq), dev, stream)
        _own(workspace, dev)
        _check(lib.dd_paged_attn(cache._ref, batch._c(T), Hq, q.data_ptr(), qs,
                                 float(scale if scale is not None else D ** -0.5), int(causal),
                                 out.data_ptr(), None if lse is None else lse.data_ptr(),
                                 workspace.data_ptr(), workspace.numel(), on.raw))
    return out, lse


def verify_draft_workspace_bytes(batch: int, total: int, vocab: int) -> int:
    return int(load().dd_verify_draft_workspace(batch, total, vocab))


def verify_draft_outputs(batch: int, total: int, device="cuda") -> dict:
    """The output tensors of verify_draft: accepted, tokens, target_prob."""
    return {"accepted": torch.empty(batch, dtype=torch.int32, device=device),
            "tokens": torch.empty(total + batch, dtype=torch.int32, device=device),
            "target_prob": torch.empty(total, dtype=torch.float32, device=device)}


def verify_draft(target_logits: torch.Tensor, draft_logits: torch.Tensor,
                 draft_tokens: torch.Tensor, draft_conf: torch.Tensor, cu_draft: torch.Tensor,
                 u_accept: torch.Tensor, u_sample: torch.Tensor, temperature: float = 1.0,
                 draft_temperature: float = 1.0, outputs: Optional[dict] = None, workspace=None,
                 stream=None) -> dict:
    """dd_verify_draft: checks drafted tokens (pred and conf of
    sample_renoise over draft_logits [T, V]) against target_logits [T + B, V]
    (sequence b's rows start at cu_draft[b] + b; one more than its drafts).
    Returns the dict of verify_draft_outputs: accepted [B], tokens [T + B]
    (accepted tokens, the next token, -1), target_prob [T]."""
    lib, dev = load(), target_logits.device
    _need(target_logits.is_cuda, "target_logits must be a CUDA tensor")
    _need(target_logits.dim() == 2 and draft_logits.dim() == 2, "logits must be 2-D")
    T, V = draft_logits.shape
    B = u_sample.numel()
    if target_logits.shape != (T + B, V):
        raise ValueError(f"target_logits: shape {tuple(target_logits.shape)}, "
                         f"expected {(T + B, V)}")
    zt, zd = target_logits.stride(), draft_logits.stride()
    if draft_logits.dtype != target_logits.dtype or draft_logits.device != dev:
        raise ValueError(f"draft_logits: {draft_logits.dtype} on {draft_logits.device}, "
                         f"expected {target_logits.dtype} on {dev}")
    if V > 1 and (zt[1] != 1 or zd[1] != 1):
        raise ValueError("a row of logits must be contiguous")
    for t, n, dt, what in ((draft_tokens, T, torch.int32, "draft_tokens"),
                           (draft_conf, T, torch.float32, "draft_conf"),
                           (cu_draft, B + 1, torch.int32, "cu_draft"),
                           (u_accept, T, torch.float32, "u_accept"),
                           (u_sample, B, torch.float32, "u_sample")):
        _dense(t, (n,), dt, dev, what)
    o = outputs
    with _on(dev, stream) as on:
        if o is None:
            o = {k: on.lend(t) for k, t in verify_draft_outputs(B, T, dev).items()}
        for name, n, dt in (("accepted", B, torch.int32), ("tokens", T + B, torch.int32),
                            ("target_prob", T, torch.float32)):
            _dense(o[name], (n,), dt, dev, name)
        if workspace is None:
            workspace = new_workspace(verify_draft_workspace_bytes(B, T, V), dev, stream)
        prm = VerifyParams(float(temperature), float(draft_temperature))
        _own(workspace, dev)
        _check(lib.dd_verify_draft(
            ctypes.byref(prm), _dtype_code(target_logits), B, T, V, target_logits.data_ptr(),
            zt[0] if T + B > 1 else V, draft_logits.data_ptr(),
            zd[0] if T > 1 else V, draft_tokens.data_ptr(),
            draft_conf.data_ptr(), cu_draft.data_ptr(), u_accept.data_ptr(), u_sample.data_ptr(),
            o["accepted"].data_ptr(), o["tokens"].data_ptr(), o["target_prob"].data_ptr(),
            workspace.data_ptr(), workspace.numel(), on.raw))
    return o


def query_device_error(workspace: torch.Tensor, stream=None):
    _check(load().dd_query_device_error(_ptr(workspace), _stream(stream)))


def set_test_stall_ns(ns: int):
    """dd_set_test_stall_ns: with ns != 0 the tensor-core kernels launched
    afterwards from this thread stall on a barrier nothing completes and
    report DD_ERR_DEVICE_TIMEOUT after ns nanoseconds (0 turns it off)."""
    load().dd_set_test_stall_ns(int(ns))


def launch_count() -> int:
    return int(load().dd_launch_count())


def reset_launch_count():
    load().dd_reset_launch_count()


def status_string(code: int) -> str:
    return load().dd_status_string(code).decode()


def last_error() -> str:
    return load().dd_last_error().decode()

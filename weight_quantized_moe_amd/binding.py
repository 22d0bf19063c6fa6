"""ctypes binding of libmoe_quant.so (argument marshalling only).

Every step of the layer runs in the HIP library; PyTorch supplies device
memory (tensors' ``data_ptr()``) and the current HIP stream.  If the library is
missing, constructing a :class:`Layer` raises: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, Optional

HERE = os.path.dirname(os.path.abspath(__file__))

ABI_VERSION = 1
FORMATS = {"int4_g128": 1, "fp8_b128": 2, "nvfp4_g16": 3}
MQ_F32, MQ_BF16 = 0, 1
SCORES = {"softmax": 0, "sigmoid": 1}
ACTIVATIONS = {"bf16": 0, "fp8": 1, "nvfp4": 2}
MQ_KV_BF16, MQ_KV_FP8 = 0, 1
GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = range(4)
STAGES = ("route", "permute", "gate_up", "down", "combine")

EXPORTED = (
    "moe_quant_init",
    "moe_quant_workspace_size",
    "moe_quant_forward",
    "moe_quant_forward_noalloc",
    "moe_quant_forward_with_router",
    "moe_quant_forward_w8a8",
    "moe_quant_forward_w4a4",
    "moe_quant_forward_gated",
    "moe_quant_gate_topk",
    "moe_quant_norm",
    "moe_quant_linear",
    "moe_quant_linear_workspace_size",
    "moe_quant_kv_append",
    "moe_quant_attend",
    "moe_quant_attend_workspace_size",
    "moe_quant_quantize_act",
    "moe_quant_quantize_act_nvfp4",
    "moe_quant_import_expert",
    "moe_quant_check",
    "moe_quant_dequantize",
    "moe_quant_router_logits",
    "moe_quant_destroy",
    "moe_quant_status_string",
    "moe_quant_last_error",
    "moe_quant_abi_version",
)


class MoeQuantError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"moe_quant status {status}: {message}")
        self.status = status


class LayerDesc(ctypes.Structure):
    _fields_ = [
        ("abi_version", ctypes.c_uint32),
        ("num_experts", ctypes.c_int32),
        ("hidden", ctypes.c_int32),
        ("intermediate", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("format", ctypes.c_int32),
        ("w13", ctypes.c_void_p),
        ("w13_scale", ctypes.c_void_p),
        ("w13_gscale", ctypes.c_void_p),
        ("w2", ctypes.c_void_p),
        ("w2_scale", ctypes.c_void_p),
        ("w2_gscale", ctypes.c_void_p),
    ]


class GateDesc(ctypes.Structure):
    _fields_ = [
        ("abi_version", ctypes.c_uint32),
        ("num_experts", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("score", ctypes.c_int32),
        ("num_groups", ctypes.c_int32),
        ("topk_groups", ctypes.c_int32),
        ("group_top", ctypes.c_int32),
        ("renormalize", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("bias", ctypes.c_void_p),
    ]


class NormDesc(ctypes.Structure):
    _fields_ = [
        ("abi_version", ctypes.c_uint32),
        ("hidden", ctypes.c_int32),
        ("residual_dtype", ctypes.c_int32),
        ("weight_dtype", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("weight_offset", ctypes.c_float),
        ("scale", ctypes.c_float),
        ("post_weight", ctypes.c_void_p),
        ("pre_weight", ctypes.c_void_p),
    ]


class LinearDesc(ctypes.Structure):
    _fields_ = [
        ("abi_version", ctypes.c_uint32),
        ("n", ctypes.c_int32),
        ("k", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("w", ctypes.c_void_p),
        ("scale", ctypes.c_void_p),
    ]


class KvCacheDesc(ctypes.Structure):
    _fields_ = [
        ("abi_version", ctypes.c_uint32),
        ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
    ]


class RotaryDesc(ctypes.Structure):
    _fields_ = [
        ("abi_version", ctypes.c_uint32),
        ("head_dim", ctypes.c_int32),
        ("rot_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("max_positions", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("cos_sin", ctypes.c_void_p),
        ("q_norm", ctypes.c_void_p),
        ("k_norm", ctypes.c_void_p),
    ]


class SrcProj(ctypes.Structure):
    _fields_ = [
        ("weight", ctypes.c_void_p),
        ("scale", ctypes.c_void_p),
        ("qzeros", ctypes.c_void_p),
        ("global_scale", ctypes.c_float),
    ]


class Probe(ctypes.Structure):
    _fields_ = [
        ("topk_ids", ctypes.c_void_p),
        ("topk_w", ctypes.c_void_p),
        ("expert_offsets", ctypes.c_void_p),
        ("sorted_token_ids", ctypes.c_void_p),
        ("inv_pos", ctypes.c_void_p),
        ("h", ctypes.c_void_p),
        ("events", ctypes.c_void_p * (2 * len(STAGES))),
    ]


def library_path() -> str:
    return os.environ.get("MOE_QUANT_LIB", os.path.join(HERE, "libmoe_quant.so"))


_LIB = None


def load_library():
    """Load libmoe_quant.so and declare its signatures (raises if missing)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise MoeQuantError(-1, f"{path} is not built; run weight_quantized_moe_amd.build.build()")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.moe_quant_init.argtypes = [ctypes.POINTER(LayerDesc), ctypes.POINTER(vp)]
    lib.moe_quant_init.restype = i32
    lib.moe_quant_workspace_size.argtypes = [vp, i64, ctypes.POINTER(sz)]
    lib.moe_quant_workspace_size.restype = i32
    lib.moe_quant_forward.argtypes = [vp, vp, i32, vp, vp, i64, vp, vp, sz,
                                      ctypes.POINTER(Probe), vp]
    lib.moe_quant_forward.restype = i32
    lib.moe_quant_forward_noalloc.argtypes = [vp, vp, i32, vp, vp, i64, vp, vp, vp]
    lib.moe_quant_forward_noalloc.restype = i32
    lib.moe_quant_forward_with_router.argtypes = [vp, vp, vp, vp, i64, vp, vp, sz, vp,
                                                  ctypes.POINTER(Probe), vp]
    lib.moe_quant_forward_with_router.restype = i32
    lib.moe_quant_import_expert.argtypes = [ctypes.POINTER(LayerDesc), i32, ctypes.POINTER(SrcProj),
                                            ctypes.POINTER(SrcProj), ctypes.POINTER(SrcProj), i32, vp, vp]
    lib.moe_quant_import_expert.restype = i32
    lib.moe_quant_forward_w8a8.argtypes = [vp, vp, i32, vp, vp, i64, vp, vp, sz, ctypes.POINTER(Probe), vp]
    lib.moe_quant_forward_w8a8.restype = i32
    lib.moe_quant_quantize_act.argtypes = [vp, i64, i32, vp, vp, vp]
    lib.moe_quant_quantize_act.restype = i32
    f32 = ctypes.c_float
    lib.moe_quant_forward_w4a4.argtypes = [vp, vp, i32, vp, vp, i64, vp, vp, sz, f32, f32,
                                           ctypes.POINTER(Probe), vp]
    lib.moe_quant_forward_w4a4.restype = i32
    lib.moe_quant_quantize_act_nvfp4.argtypes = [vp, i64, i32, f32, vp, vp, vp]
    lib.moe_quant_quantize_act_nvfp4.restype = i32
    lib.moe_quant_check.argtypes = [vp, vp, vp]
    lib.moe_quant_check.restype = i32
    lib.moe_quant_dequantize.argtypes = [vp, i32, i32, vp, vp]
    lib.moe_quant_dequantize.restype = i32
    lib.moe_quant_router_logits.argtypes = [vp, vp, i64, i32, i32, vp, vp]
    lib.moe_quant_router_logits.restype = i32
    lib.moe_quant_gate_topk.argtypes = [ctypes.POINTER(GateDesc), vp, i32, i64, vp, vp, vp]
    lib.moe_quant_gate_topk.restype = i32
    lib.moe_quant_forward_gated.argtypes = [vp, ctypes.POINTER(GateDesc), vp, i32, vp, vp, vp, i64, vp, vp, sz, i32,
                                            f32, f32, vp, ctypes.POINTER(Probe), vp]
    lib.moe_quant_forward_gated.restype = i32
    lib.moe_quant_norm.argtypes = [ctypes.POINTER(NormDesc), vp, vp, vp, i32, i32, i64, vp, vp, vp]
    lib.moe_quant_norm.restype = i32
    lib.moe_quant_linear_workspace_size.argtypes = [ctypes.POINTER(LinearDesc), i64, ctypes.POINTER(sz)]
    lib.moe_quant_linear_workspace_size.restype = i32
    lib.moe_quant_linear.argtypes = [ctypes.POINTER(LinearDesc), vp, vp, i64, vp, vp, sz, vp]
    lib.moe_quant_linear.restype = i32
    lib.moe_quant_kv_append.argtypes = [ctypes.POINTER(KvCacheDesc), ctypes.POINTER(RotaryDesc), i32, vp, i64, vp, i64,
                                        vp, i64, vp, vp, i64, vp, vp]
    lib.moe_quant_kv_append.restype = i32
    lib.moe_quant_attend_workspace_size.argtypes = [ctypes.POINTER(KvCacheDesc), i32, i64, ctypes.POINTER(sz)]
    lib.moe_quant_attend_workspace_size.restype = i32
    lib.moe_quant_attend.argtypes = [ctypes.POINTER(KvCacheDesc), i32, f32, i32, vp, vp, i64, i32, vp, i64, vp, vp, vp,
                                     sz, vp]
    lib.moe_quant_attend.restype = i32
    lib.moe_quant_destroy.argtypes = [vp]
    lib.moe_quant_destroy.restype = None
    lib.moe_quant_status_string.argtypes = [i32]
    lib.moe_quant_status_string.restype = ctypes.c_char_p
    lib.moe_quant_last_error.argtypes = []
    lib.moe_quant_last_error.restype = ctypes.c_char_p
    lib.moe_quant_abi_version.argtypes = []
    lib.moe_quant_abi_version.restype = ctypes.c_uint32
    if lib.moe_quant_abi_version() != ABI_VERSION:
        raise MoeQuantError(7, "library ABI version differs from the binding's")
    _LIB = lib
    return lib


def _check(lib, status: int):
    if status != 0:
        raise MoeQuantError(status, lib.moe_quant_last_error().decode())


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _need(t, name, shape, dtypes, device=None):
    """Raise ValueError unless tensor ``t`` is contiguous, of the given shape
    (None entries match any size) and one of ``dtypes``.  Checked before any
    launch: a wrong shape or a strided view would otherwise become
    out-of-bounds device accesses.  (``device`` is checked by _on_gpu.)"""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.dim() != len(shape) or any(s is not None and s != d for s, d in zip(shape, t.shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_gpu(device, **tensors):
    """Raise ValueError unless every given tensor is a GPU tensor on ``device``
    (the first one's device if ``device`` is None)."""
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        device = device if device is not None else t.device
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


class _Quick:
    """What the calls of the gate and the norm look up once: small calls are bound
    by the host, so their checks take the form that costs the least, in front of
    _need and _on_gpu (which name what is wrong)."""

    def __init__(self):
        import torch
        self.device_now = torch.cuda.current_device
        self.raw_stream = torch._C._cuda_getCurrentRawStream     # of a GPU index
        self.f32, self.bf16, self.i32, self.u8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
        self.on = torch.cuda.device


_quick = None


def _get_quick() -> _Quick:
    global _quick
    if _quick is None:
        _quick = _Quick()
    return _quick


def _fits(t, shape, dtype, index) -> bool:
    """Whether ``t`` is a contiguous tensor of this shape and dtype on GPU ``index``."""
    return t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == index


def _empty(shape, dtype, device, stream):
    """A new tensor for work on ``stream`` (None: the current one): taken from that
    stream's memory, so no earlier tensor's work on another stream still uses it."""
    import torch
    if stream is None or not device.type == "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def router_logits(hidden, router_w, out=None, stream=None):
    """Router logits float32 [T, E] = hidden [T, H] . router_w [E, H]^T, both
    bfloat16 on the GPU (moe_quant_router_logits)."""
    import torch
    lib = load_library()
    if hidden.dim() != 2 or router_w.dim() != 2:
        raise ValueError("need hidden [T, H] and router weight [E, H]")
    t, h = hidden.shape
    e = router_w.shape[0]
    _need(hidden, "hidden", (t, h), (torch.bfloat16,))
    _need(router_w, "router_w", (e, h), (torch.bfloat16,))
    if out is None:
        out = torch.empty((t, e), dtype=torch.float32, device=hidden.device)
    _need(out, "out", (t, e), (torch.float32,))
    _on_gpu(None, hidden=hidden, router_w=router_w, out=out)
    _check(lib, lib.moe_quant_router_logits(_ptr(hidden), _ptr(router_w), t, h, e, _ptr(out),
                                            _stream(stream)))
    return out


def import_expert(fmt: str, dst, expert: int, gate, up, down, gptq_zero_offset: int = 1,
                  bad_zero_points=None, stream=None):
    """Write one expert's checkpoint tensors into packed layer buffers
    (moe_quant_import_expert).  ``dst`` = (w13, w13_scale, w2, w2_scale,
    w13_gscale, w2_gscale) GPU tensors in the library layouts (gscales None
    except for NVFP4).  ``gate``/``up``/``down`` per format: FP8 (weight uint8
    [N, K], weight_scale_inv float32 [N/128, K/128]); INT4 auto_gptq (qweight
    int32 [K/8, N], qzeros int32 [K/128, N/8], scales float16 [K/128, N]);
    NVFP4 compressed-tensors (weight_packed uint8 [N, K/2], weight_scale
    uint8 [N, K/16], weight_global_scale float)."""
    import torch
    lib = load_library()
    w13, s13, w2, s2, g13, g2 = dst
    e, n13, _ = w13.shape
    h = w2.shape[1]
    i = n13 // 2
    kdiv = 1 if fmt == "fp8_b128" else 2
    _need(w13, "w13", (e, 2 * i, h // kdiv), (torch.uint8,))
    _need(w2, "w2", (e, h, i // kdiv), (torch.uint8,))

    def src(p, n, k, name):
        if fmt == "fp8_b128":
            w, s = p
            _need(w, f"{name}.weight", (n, k), (torch.uint8,))
            _need(s, f"{name}.weight_scale_inv", (n // 128, k // 128), (torch.float32,))
            _on_gpu(w13.device, w=w, s=s)
            return SrcProj(w.data_ptr(), s.data_ptr(), None, 0.0)
        if fmt == "int4_g128":
            qw, qz, sc = p
            _need(qw, f"{name}.qweight", (k // 8, n), (torch.int32,))
            _need(qz, f"{name}.qzeros", (k // 128, n // 8), (torch.int32,))
            _need(sc, f"{name}.scales", (k // 128, n), (torch.float16,))
            _on_gpu(w13.device, qw=qw, qz=qz, sc=sc)
            return SrcProj(qw.data_ptr(), sc.data_ptr(), qz.data_ptr(), 0.0)
        wp, ws, g = p
        _need(wp, f"{name}.weight_packed", (n, k // 2), (torch.uint8,))
        _need(ws, f"{name}.weight_scale", (n, k // 16), (torch.uint8,))
        _on_gpu(w13.device, wp=wp, ws=ws)
        return SrcProj(wp.data_ptr(), ws.data_ptr(), None, float(g))

    sg, su, sd = src(gate, i, h, "gate_proj"), src(up, i, h, "up_proj"), src(down, h, i, "down_proj")
    d = LayerDesc(ABI_VERSION, e, h, i, 1, FORMATS[fmt], _ptr(w13), _ptr(s13), _ptr(g13),
                  _ptr(w2), _ptr(s2), _ptr(g2))
    if bad_zero_points is not None:
        _need(bad_zero_points, "bad_zero_points", (1,), (torch.int32,))
    _check(lib, lib.moe_quant_import_expert(ctypes.byref(d), expert, ctypes.byref(sg), ctypes.byref(su),
                                            ctypes.byref(sd), gptq_zero_offset, _ptr(bad_zero_points),
                                            _stream(stream)))


def quantize_act(x, codes=None, scales=None, stream=None):
    """Dynamic 1x128 FP8 quantization of float32 rows x [rows, K] on the GPU
    (moe_quant_quantize_act): returns (codes uint8 [rows, K], scales float32
    [rows, K/128])."""
    import torch
    lib = load_library()
    if x.dim() != 2:
        raise ValueError("x must be [rows, K]")
    r, k = x.shape
    _need(x, "x", (r, k), (torch.float32,))
    if codes is None:
        codes = torch.empty((r, k), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((r, k // 128), dtype=torch.float32, device=x.device)
    _need(codes, "codes", (r, k), (torch.uint8,))
    _need(scales, "scales", (r, k // 128), (torch.float32,))
    _on_gpu(None, x=x, codes=codes, scales=scales)
    _check(lib, lib.moe_quant_quantize_act(_ptr(x), r, k, _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def quantize_act_nvfp4(x, gscale: float, codes=None, scales=None, stream=None):
    """NVFP4 quantization of float32 rows x [rows, K] with global scale
    ``gscale`` on the GPU (moe_quant_quantize_act_nvfp4): returns (codes uint8
    [rows, K/2], two E2M1 codes per byte, even k in the low nibble; E4M3 block
    scales uint8 [rows, K/16])."""
    import torch
    lib = load_library()
    if x.dim() != 2:
        raise ValueError("x must be [rows, K]")
    r, k = x.shape
    _need(x, "x", (r, k), (torch.float32,))
    if codes is None:
        codes = torch.empty((r, k // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((r, k // 16), dtype=torch.uint8, device=x.device)
    _need(codes, "codes", (r, k // 2), (torch.uint8,))
    _need(scales, "scales", (r, k // 16), (torch.uint8,))
    _on_gpu(None, x=x, codes=codes, scales=scales)
    _check(lib, lib.moe_quant_quantize_act_nvfp4(_ptr(x), r, k, float(gscale), _ptr(codes), _ptr(scales),
                                                 _stream(stream)))
    return codes, scales


def _mq_dtype(dtype) -> int:
    import torch
    return MQ_F32 if dtype == torch.float32 else MQ_BF16


class Gate:
    """The gate of a routed layer (mq_gate): softmax or sigmoid scores, a balance
    ``bias`` (float32 [E] on the GPU) that takes part in the selection only,
    ``topk_groups`` of ``num_groups`` groups ranked by their ``group_top`` (1 or
    2) largest selection scores, top-k, renormalised or raw weights, times
    ``scale``.  The bias must stay alive as long as the gate."""

    def __init__(self, num_experts: int, top_k: int, score: str = "softmax", bias=None,
                 num_groups: int = 1, topk_groups: int = 1, group_top: int = 1,
                 renormalize: bool = True, scale: float = 1.0):
        import torch
        self._lib = load_library()
        if score not in SCORES:
            raise ValueError(f"unknown score {score!r}")
        if bias is not None:
            _need(bias, "bias", (num_experts,), (torch.float32,))
            _on_gpu(None, bias=bias)
        self.num_experts, self.top_k, self.bias = num_experts, top_k, bias
        self._q, self._call = _get_quick(), self._lib.moe_quant_gate_topk
        self._bias_index = None if bias is None else bias.get_device()
        self.desc = GateDesc(ABI_VERSION, num_experts, top_k, SCORES[score], num_groups, topk_groups,
                             group_top, int(renormalize), scale, _ptr(bias))
        self._ref = ctypes.byref(self.desc)
        # the library's own checks of the fields; no tokens, so nothing is enqueued
        _check(self._lib, self._lib.moe_quant_gate_topk(self._ref, None, MQ_F32, 0, None,
                                                        None, None))

    def topk(self, logits, ids=None, weights=None, stream=None):
        """The gate of logits [T, E] (float32 or bfloat16): returns (ids int32
        [T, k], weights float32 [T, k])."""
        q, given, index, dtype = self._q, logits.shape, logits.get_device(), logits.dtype
        if len(given) != 2:
            raise ValueError("logits must be [T, E]")
        t, e = given[0], self.num_experts
        shape = (t, self.top_k)
        if index >= 0 and index != q.device_now():
            with q.on(index):
                return self.topk(logits, ids, weights, stream)
        if ids is None:
            ids = _empty(shape, q.i32, logits.device, stream)
        if weights is None:
            weights = _empty(shape, q.f32, logits.device, stream)
        if not (index >= 0 and (dtype is q.f32 or dtype is q.bf16) and given[1] == e and logits.is_contiguous()
                and ids.dtype is q.i32 and ids.shape == shape and ids.is_contiguous() and ids.get_device() == index
                and weights.dtype is q.f32 and weights.shape == shape and weights.is_contiguous()
                and weights.get_device() == index and self._bias_index in (None, index)):
            _need(logits, "logits", (t, e), (q.f32, q.bf16))
            _need(ids, "ids", shape, (q.i32,))
            _need(weights, "weights", shape, (q.f32,))
            _on_gpu(logits.device, logits=logits, bias=self.bias, ids=ids, weights=weights)
        st = self._call(self._ref, logits.data_ptr(), MQ_F32 if dtype is q.f32 else MQ_BF16, t, ids.data_ptr(),
                        weights.data_ptr(), q.raw_stream(index) if stream is None else stream.cuda_stream)
        if st:
            _check(self._lib, st)
        return ids, weights


class ResidualNorm:
    """Norms before and after a block with its gate, the residual scale and the
    residual add in one pass (moe_quant_norm).

    ``post_weight`` [H]: norm of the block's output (None: none); ``pre_weight``
    [H]: norm of the new residual, the next block's input (None: none); both
    float32 or both bfloat16, on the GPU, alive as long as the object.
    ``weight_offset`` is 1 where weights are stored as w - 1."""

    def __init__(self, hidden: int, post_weight=None, pre_weight=None, eps: float = 1e-6,
                 weight_offset: float = 0.0, scale: float = 1.0, residual_dtype=None):
        import torch
        self._lib = load_library()
        residual_dtype = residual_dtype or torch.bfloat16
        types = (torch.float32, torch.bfloat16)
        if residual_dtype not in types:
            raise ValueError(f"residual_dtype {residual_dtype}, expected one of {types}")
        weight_dtype = torch.bfloat16
        for name, w in (("post_weight", post_weight), ("pre_weight", pre_weight)):
            if w is not None:
                _need(w, name, (hidden,), types)
                weight_dtype = w.dtype
        if post_weight is not None and pre_weight is not None and post_weight.dtype != pre_weight.dtype:
            raise ValueError("post_weight and pre_weight must have one dtype")
        _on_gpu(None, post_weight=post_weight, pre_weight=pre_weight)
        self.hidden, self.residual_dtype = hidden, residual_dtype
        self.post_weight, self.pre_weight = post_weight, pre_weight
        self._types, self._q, self._call = types, _get_quick(), self._lib.moe_quant_norm
        self._index = frozenset(w.get_device() for w in (post_weight, pre_weight) if w is not None)
        self.desc = NormDesc(ABI_VERSION, hidden, _mq_dtype(residual_dtype), _mq_dtype(weight_dtype), eps,
                             weight_offset, scale, _ptr(post_weight), _ptr(pre_weight))
        self._ref = ctypes.byref(self.desc)
        # the library's own checks of the fields; no tokens, so nothing is enqueued
        _check(self._lib, self._lib.moe_quant_norm(self._ref, None, None, None, GATE_NONE, 0, 0,
                                                   None, None, None))

    def forward(self, x=None, residual=None, gate=None, residual_out=None, norm_out=None, stream=None):
        """``x`` bfloat16 [T, H] (the block's output), ``residual`` [T, H], ``gate``
        float32 or bfloat16: [H] per channel, [T, 1] per token or [T, H].
        Returns (residual_out, norm_out); norm_out is None without a
        ``pre_weight``.  The outputs may be the inputs' own buffers."""
        q, first = self._q, residual if x is None else x
        given = None if first is None else first.shape
        if given is None or len(given) != 2:
            raise ValueError("need x or residual [T, H]")
        t, h, index = given[0], self.hidden, first.get_device()
        if index >= 0 and index != q.device_now():
            with q.on(index):
                return self.forward(x, residual, gate, residual_out, norm_out, stream)
        shape, rd, bf16 = (t, h), self.residual_dtype, q.bf16
        kind, gate_dtype, gate_ptr = GATE_NONE, MQ_F32, None
        if gate is not None:
            gs = gate.shape
            kind = (GATE_CHANNEL if gs == (h,) else GATE_TOKEN if gs == (t, 1) else GATE_FULL if gs == shape else None)
            if kind is None:
                raise ValueError(f"gate has shape {tuple(gs)}, expected ({h},), ({t}, 1) or ({t}, {h})")
            gate_dtype, gate_ptr = _mq_dtype(gate.dtype), gate.data_ptr()
        if residual_out is None:
            residual_out = _empty(shape, rd, first.device, stream)
        if self.pre_weight is None:
            if norm_out is not None:
                raise ValueError("norm_out needs a pre_weight")
        elif norm_out is None:
            norm_out = _empty(shape, bf16, first.device, stream)
        if not (index >= 0 and self._index <= {index}
                and (x is None or x.dtype is bf16 and x.shape == shape and x.is_contiguous() and x.get_device() == index)
                and (residual is None or residual.dtype is rd and residual.shape == shape and residual.is_contiguous()
                     and residual.get_device() == index)
                and residual_out.dtype is rd and residual_out.shape == shape and residual_out.is_contiguous()
                and residual_out.get_device() == index
                and (norm_out is None or norm_out.dtype is bf16 and norm_out.shape == shape and norm_out.is_contiguous()
                     and norm_out.get_device() == index)
                and (gate is None or gate.dtype in self._types and gate.is_contiguous() and gate.get_device() == index)):
            if x is not None:
                _need(x, "x", shape, (bf16,))
            if residual is not None:
                _need(residual, "residual", shape, (rd,))
            if gate is not None:
                _need(gate, "gate", tuple(gs), self._types)
            _need(residual_out, "residual_out", shape, (rd,))
            if norm_out is not None:
                _need(norm_out, "norm_out", shape, (bf16,))
            _on_gpu(first.device, x=x, residual=residual, gate=gate, residual_out=residual_out, norm_out=norm_out,
                    post_weight=self.post_weight, pre_weight=self.pre_weight)
        st = self._call(
            self._ref, None if x is None else x.data_ptr(), None if residual is None else residual.data_ptr(), gate_ptr,
            kind, gate_dtype, t, residual_out.data_ptr(), None if norm_out is None else norm_out.data_ptr(),
            q.raw_stream(index) if stream is None else stream.cuda_stream)
        if st:
            _check(self._lib, st)
        return residual_out, norm_out


class Linear:
    """A dense projection on E4M3 weights with a scale for each block of 128
    (moe_quant_linear): ``w`` uint8 [N, K] (E4M3FN bits), ``w_scale`` float32
    [ceil(N / 128), ceil(K / 128)], both on the GPU and alive as long as the object.
    The rows are quantized to E4M3 per 128 values; their scale is a product with
    1 / 448 where ``Layer.forward_w8a8`` divides, so one code in 900 is not its code.
    ``out_dtype``: bfloat16 (default) or float32."""

    def __init__(self, w, w_scale, out_dtype=None):
        import torch
        self._lib = load_library()
        out_dtype = out_dtype or torch.bfloat16
        if out_dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"out_dtype {out_dtype}, expected float32 or bfloat16")
        if w.dim() != 2:
            raise ValueError("w must be [N, K]")
        n, k = w.shape
        _need(w, "w", (n, k), (torch.uint8,))
        _need(w_scale, "w_scale", (-(-n // 128), -(-k // 128)), (torch.float32,))
        _on_gpu(None, w=w, w_scale=w_scale)
        self.n, self.k, self.out_dtype, self.device = n, k, out_dtype, w.device
        self._keep = (w, w_scale)
        self._q, self._call, self._index = _get_quick(), self._lib.moe_quant_linear, w.get_device()
        self.desc = LinearDesc(ABI_VERSION, min(n, 2 ** 31 - 1), min(k, 2 ** 31 - 1), _mq_dtype(out_dtype), _ptr(w),
                               _ptr(w_scale))
        self._ref = ctypes.byref(self.desc)
        self._last_need = (-1, 0)      # (tokens, bytes) of the last call
        self.workspace_size(0)         # the library's own checks of the fields

    def workspace_size(self, num_tokens: int) -> int:
        b = ctypes.c_size_t()
        _check(self._lib, self._lib.moe_quant_linear_workspace_size(self._ref, num_tokens, ctypes.byref(b)))
        return b.value

    def _workspace_need(self, num_tokens: int) -> int:
        last = self._last_need
        if last[0] != num_tokens:
            last = self._last_need = (num_tokens, self.workspace_size(num_tokens))
        return last[1]

    def workspace(self, num_tokens: int):
        import torch
        return torch.empty(max(self.workspace_size(num_tokens), 256), dtype=torch.uint8, device=self.device)

    def forward(self, x, residual=None, out=None, workspace=None, stream=None):
        """``x`` bfloat16 [T, K] -> ``out`` [T, N] = x w^T (+ ``residual``, bfloat16
        [T, N], which may be ``out`` itself where that is bfloat16)."""
        q, given, index = self._q, x.shape, self._index
        if len(given) != 2:
            raise ValueError("x must be [T, K]")
        t = given[0]
        if index != q.device_now():
            with q.on(index):
                return self.forward(x, residual, out, workspace, stream)
        shape, bf16 = (t, self.n), q.bf16
        if out is None:
            out = _empty(shape, self.out_dtype, self.device, stream)
        if workspace is None:
            workspace = _empty((max(self._workspace_need(t), 256),), q.u8, self.device, stream)
        if not (_fits(x, (t, self.k), bf16, index) and _fits(out, shape, self.out_dtype, index)
                and (residual is None or _fits(residual, shape, bf16, index))
                and workspace.is_contiguous() and workspace.get_device() == index):
            _need(x, "x", (t, self.k), (bf16,))
            if residual is not None:
                _need(residual, "residual", shape, (bf16,))
            _need(out, "out", shape, (self.out_dtype,))
            if not workspace.is_contiguous():
                raise ValueError("workspace must be contiguous")
            _on_gpu(self.device, x=x, residual=residual, out=out, workspace=workspace)
        st = self._call(self._ref, x.data_ptr(), None if residual is None else residual.data_ptr(), t, out.data_ptr(),
                        workspace.data_ptr(), _nbytes(workspace),
                        q.raw_stream(index) if stream is None else stream.cuda_stream)
        if st:
            _check(self._lib, st)
        return out


class Rotary:
    """What happens to a head's query and key before attention (mq_rotary): the
    per-head RMS norm (``q_norm``, ``k_norm`` bfloat16 [D], None: none) and the
    rotation by the position's angles: ``cos_sin`` float32 [positions, R], the R / 2
    cosines and then the sines of each position (None: no rotation), R a multiple
    of 16 up to D; pairs (i, i + R / 2), or (2i, 2i + 1) if ``interleaved``.  All on
    the GPU, alive as long as the object."""

    def __init__(self, head_dim: int, cos_sin=None, interleaved: bool = False, q_norm=None, k_norm=None,
                 eps: float = 1e-6):
        import torch
        if cos_sin is not None:
            if cos_sin.dim() != 2:
                raise ValueError("cos_sin must be [positions, R]")
            _need(cos_sin, "cos_sin", tuple(cos_sin.shape), (torch.float32,))
            if not 0 < cos_sin.shape[1] <= head_dim or cos_sin.shape[1] % 16:
                raise ValueError(f"cos_sin has {cos_sin.shape[1]} columns, expected a multiple of 16 up to {head_dim}")
            if cos_sin.shape[0] < 1:
                raise ValueError("cos_sin has no positions")
        for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
            if w is not None:
                _need(w, name, (head_dim,), (torch.bfloat16,))
        _on_gpu(None, cos_sin=cos_sin, q_norm=q_norm, k_norm=k_norm)
        self.head_dim, self.rotates = head_dim, cos_sin is not None
        self._keep = (cos_sin, q_norm, k_norm)
        self._index = frozenset(w.get_device() for w in self._keep if w is not None)
        p, r = cos_sin.shape if self.rotates else (0, 0)
        self.desc = RotaryDesc(ABI_VERSION, head_dim, r, int(interleaved), min(p, 2 ** 31 - 1), eps, _ptr(cos_sin),
                               _ptr(q_norm), _ptr(k_norm))
        self._ref = ctypes.byref(self.desc)

    @staticmethod
    def table(positions: int, rot_dim: int, base: float = 10000.0, device="cuda"):
        """cos_sin of the angles position * base^(-2i / rot_dim), computed in 64 bits."""
        import torch
        rate = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
        angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * rate
        return torch.cat((angle.cos(), angle.sin()), 1).float()


class KVCache:
    """A paged cache of keys and values (mq_kv_cache): ``k`` and ``v`` [pages,
    kv_heads, page_size, D], bfloat16 or float8_e4m3fn (then a key is its E4M3
    value times ``k_scale``, a value times ``v_scale``), on the GPU, alive as long
    as the object.  Slot p * page_size + s is token s of page p."""

    def __init__(self, k, v, k_scale: float = 1.0, v_scale: float = 1.0):
        import torch
        self._lib = load_library()
        if k.dim() != 4:
            raise ValueError("k must be [pages, kv_heads, page_size, D]")
        _need(k, "k", tuple(k.shape), (torch.bfloat16, torch.float8_e4m3fn))
        _need(v, "v", tuple(k.shape), (k.dtype,))
        _on_gpu(None, k=k, v=v)
        pages, heads, page_size, d = k.shape
        self.k, self.v, self.device = k, v, k.device
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page_size, d
        self._q, self._index = _get_quick(), k.get_device()
        self._append, self._attend = self._lib.moe_quant_kv_append, self._lib.moe_quant_attend
        self.desc = KvCacheDesc(ABI_VERSION, heads, d, page_size, pages,
                                MQ_KV_BF16 if k.dtype == torch.bfloat16 else MQ_KV_FP8, k_scale, v_scale, _ptr(k),
                                _ptr(v))
        self._ref = ctypes.byref(self.desc)
        self._last_need = (None, 0)             # (batch and query heads, bytes) of the last attend
        self.attend_workspace_size(0, heads)    # the library's own checks of the fields

    def _heads(self, t, name, tokens, heads):
        """Token stride of ``t`` [T, heads, D]: heads side by side, tokens any number of values apart."""
        d = self.head_dim
        step, hs, ds = t.stride()
        if not (t.dtype is self._q.bf16 and t.shape == (tokens, heads, d) and t.get_device() == self._index and ds == 1
                and (hs == d or heads == 1)):
            if t.dtype is not self._q.bf16:
                raise ValueError(f"{name} has dtype {t.dtype}, expected {self._q.bf16}")
            if t.shape != (tokens, heads, d):
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(tokens, heads, d)}")
            _on_gpu(self.device, **{name: t})
            raise ValueError(f"the heads of {name} must lie one behind the other")
        return step if tokens > 1 else heads * d

    def append(self, rotary, q, k, v, positions, slots, q_out=None, stream=None):
        """Norm and rotate ``q`` bfloat16 [T, q_heads, D] (None: no queries) and ``k``
        [T, kv_heads, D], and write ``k`` and ``v`` into their ``slots`` (int32 [T];
        negative: padding, nothing of the token is written).  ``positions`` int32
        [T] (not used without a rotation).  The heads of a token lie side by side, tokens
        any multiple of 8 values apart, so all three may be views of one fused
        projection.  Returns ``q_out`` [T, q_heads, D] (None without queries)."""
        if k.dim() != 3 or v.dim() != 3:
            raise ValueError("k and v must be [T, kv_heads, D]")
        w, index, t = self._q, self._index, k.shape[0]
        if index != w.device_now():
            with w.on(index):
                return self.append(rotary, q, k, v, positions, slots, q_out, stream)
        ks, vs = self._heads(k, "k", t, self.kv_heads), self._heads(v, "v", t, self.kv_heads)
        hq, qs, qp, op = 0, 0, None, None
        if q is not None:
            if q.dim() != 3:
                raise ValueError("q must be [T, q_heads, D]")
            hq = q.shape[1]
            qs, qp = self._heads(q, "q", t, hq), q.data_ptr()
            shape = (t, hq, self.head_dim)
            if q_out is None:
                q_out = _empty(shape, w.bf16, self.device, stream)
            elif not _fits(q_out, shape, w.bf16, index):
                _need(q_out, "q_out", shape, (w.bf16,))
                _on_gpu(self.device, q_out=q_out)
            op = q_out.data_ptr()
        elif q_out is not None:
            raise ValueError("q_out needs q")
        pp = None
        if rotary.rotates:
            if positions is None or not _fits(positions, (t,), w.i32, index):
                _need(positions, "positions", (t,), (w.i32,))
                _on_gpu(self.device, positions=positions)
            pp = positions.data_ptr()
        if not _fits(slots, (t,), w.i32, index):
            _need(slots, "slots", (t,), (w.i32,))
            _on_gpu(self.device, slots=slots)
        if not rotary._index <= {index}:
            _on_gpu(self.device, **dict(zip(("cos_sin", "q_norm", "k_norm"), rotary._keep)))
        st = self._append(self._ref, rotary._ref, hq, qp, qs, k.data_ptr(), ks, v.data_ptr(), vs, pp, slots.data_ptr(), t,
                          op, w.raw_stream(index) if stream is None else stream.cuda_stream)
        if st:
            _check(self._lib, st)
        return q_out

    def attend_workspace_size(self, batch: int, q_heads: int) -> int:
        b = ctypes.c_size_t()
        _check(self._lib, self._lib.moe_quant_attend_workspace_size(self._ref, q_heads, batch, ctypes.byref(b)))
        return b.value

    def _attend_need(self, batch: int, q_heads: int) -> int:
        last, what = self._last_need, (batch, q_heads)
        if last[0] != what:
            last = self._last_need = (what, self.attend_workspace_size(batch, q_heads))
        return last[1]

    def attend_workspace(self, batch: int, q_heads: int):
        import torch
        return torch.empty(max(self.attend_workspace_size(batch, q_heads), 256), dtype=torch.uint8, device=self.device)

    def attend(self, q, block_table, lengths, scale: Optional[float] = None, window: int = 0, out=None, lse=None,
               workspace=None, stream=None):
        """Attention of one new token of each request (moe_quant_attend): ``q``
        bfloat16 [B, q_heads, D] over the first ``lengths`` (int32 [B]) tokens of
        the pages in ``block_table`` (int32 [B, pages], rows any distance apart),
        the last ``window`` of them if that is not 0.  ``scale``: D^-1/2 if None.
        Returns ``out`` (bfloat16 [B, q_heads, D]; may be ``q``); ``lse`` (float32
        [B, q_heads]) receives the logarithms of the exponentials' sums."""
        if q.dim() != 3:
            raise ValueError("q must be [B, q_heads, D]")
        w, index = self._q, self._index
        b, hq, d = q.shape
        if index != w.device_now():
            with w.on(index):
                return self.attend(q, block_table, lengths, scale, window, out, lse, workspace, stream)
        shape = (b, hq, self.head_dim)
        if out is None:
            out = _empty(shape, w.bf16, self.device, stream)
        if workspace is None:
            workspace = _empty((max(self._attend_need(b, hq), 256),), w.u8, self.device, stream)
        if block_table.dim() != 2 or block_table.shape[0] != b or (block_table.shape[1] > 1
                                                                   and block_table.stride(1) != 1):
            raise ValueError(f"block_table must be [{b}, pages], the pages of a request side by side")
        pages = block_table.shape[1]
        apart = block_table.stride(0) if b > 1 else pages
        if not (_fits(q, shape, w.bf16, index) and _fits(out, shape, w.bf16, index)
                and block_table.dtype is w.i32 and block_table.get_device() == index
                and _fits(lengths, (b,), w.i32, index) and (lse is None or _fits(lse, (b, hq), w.f32, index))
                and workspace.is_contiguous() and workspace.get_device() == index and apart >= pages):
            _need(q, "q", shape, (w.bf16,))
            _need(out, "out", shape, (w.bf16,))
            if block_table.dtype is not w.i32:
                raise ValueError(f"block_table has dtype {block_table.dtype}, expected {w.i32}")
            if apart < pages:
                raise ValueError("the rows of block_table must not overlap")
            _need(lengths, "lengths", (b,), (w.i32,))
            if lse is not None:
                _need(lse, "lse", (b, hq), (w.f32,))
            if not workspace.is_contiguous():
                raise ValueError("workspace must be contiguous")
            _on_gpu(self.device, q=q, out=out, block_table=block_table, lengths=lengths, lse=lse, workspace=workspace)
        if not (0 <= window < 2 ** 31 and pages < 2 ** 31):     # ctypes would pass their low 32 bits on
            window, pages = -1 if window < 0 else min(window, 2 ** 31 - 1), min(pages, 2 ** 31 - 1)
        st = self._attend(self._ref, hq, d ** -0.5 if scale is None else scale, window, q.data_ptr(),
                          block_table.data_ptr(), apart, pages, lengths.data_ptr(), b, out.data_ptr(),
                          None if lse is None else lse.data_ptr(), workspace.data_ptr(), _nbytes(workspace),
                          w.raw_stream(index) if stream is None else stream.cuda_stream)
        if st:
            _check(self._lib, st)
        return out


class Layer:
    """One MoE expert layer over packed weights resident on the GPU.

    ``w13`` [E, 2I, H/2] (4-bit formats) or [E, 2I, H] (FP8) uint8, ``w2``
    [E, H, I/2] or [E, H, I]; scales and global scales as documented in
    ``include/moe_quant.h``.  All tensors must live on the GPU and stay alive
    as long as the layer.
    """

    def __init__(self, fmt: str, w13, w13_scale, w2, w2_scale, top_k: int,
                 w13_gscale=None, w2_gscale=None):
        self._lib = load_library()
        if fmt not in FORMATS:
            raise ValueError(f"unknown format {fmt!r}")
        self.fmt = fmt
        import torch
        if w13.dim() != 3 or w2.dim() != 3:
            raise ValueError("w13 and w2 must be [E, N, K-bytes] tensors")
        e, n13, kb = w13.shape
        e2, h, _ = w2.shape
        if e2 != e:
            raise ValueError("w13 and w2 disagree on the number of experts")
        i = n13 // 2
        kdiv = 1 if fmt == "fp8_b128" else 2
        u8 = (torch.uint8,)
        _need(w13, "w13", (e, 2 * i, h // kdiv), u8)
        _need(w2, "w2", (e, h, i // kdiv), u8)
        if fmt == "int4_g128":
            _need(w13_scale, "w13_scale", (e, 2 * i, h // 128), (torch.float16,))
            _need(w2_scale, "w2_scale", (e, h, i // 128), (torch.float16,))
        elif fmt == "fp8_b128":
            _need(w13_scale, "w13_scale", (e, 2 * i // 128, h // 128), (torch.float32,))
            _need(w2_scale, "w2_scale", (e, h // 128, i // 128), (torch.float32,))
        else:
            _need(w13_scale, "w13_scale", (e, 2 * i, h // 16), u8)
            _need(w2_scale, "w2_scale", (e, h, i // 16), u8)
            _need(w13_gscale, "w13_gscale", (e,), (torch.float32,))
            _need(w2_gscale, "w2_gscale", (e,), (torch.float32,))
        _on_gpu(None, w13=w13, w13_scale=w13_scale, w2=w2, w2_scale=w2_scale,
                w13_gscale=w13_gscale, w2_gscale=w2_gscale)
        self.device = w13.device
        self.num_experts, self.hidden, self.inter, self.top_k = e, h, n13 // 2, top_k
        self._keep = (w13, w13_scale, w2, w2_scale, w13_gscale, w2_gscale)
        d = LayerDesc(ABI_VERSION, e, h, n13 // 2, top_k, FORMATS[fmt],
                      _ptr(w13), _ptr(w13_scale), _ptr(w13_gscale),
                      _ptr(w2), _ptr(w2_scale), _ptr(w2_gscale))
        handle = ctypes.c_void_p()
        _check(self._lib, self._lib.moe_quant_init(ctypes.byref(d), ctypes.byref(handle)))
        self._h = handle

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self._lib.moe_quant_destroy(h)
            self._h = None

    def workspace_size(self, num_tokens: int) -> int:
        n = ctypes.c_size_t()
        _check(self._lib, self._lib.moe_quant_workspace_size(self._h, num_tokens, ctypes.byref(n)))
        return n.value

    _last_need = (-1, 0)      # (tokens, bytes) of the last gated forward

    def _workspace_need(self, num_tokens: int) -> int:
        last = self._last_need
        if last[0] != num_tokens:
            last = self._last_need = (num_tokens, self.workspace_size(num_tokens))
        return last[1]

    def workspace(self, num_tokens: int, device=None):
        import torch
        return torch.empty(max(self.workspace_size(num_tokens), 256), dtype=torch.uint8,
                           device=device or self.device)

    def forward(self, logits, hidden, residual=None, out=None, workspace=None,
                probe: Optional[Dict] = None, events=None, stream=None):
        """Enqueue one forward from router logits; returns ``out`` (bfloat16 [T, H])."""
        return self._forward(logits, None, hidden, residual, out, workspace, probe, events,
                             stream, None)

    def forward_w8a8(self, logits, hidden, residual=None, out=None, workspace=None,
                     probe: Optional[Dict] = None, events=None, stream=None):
        """W8A8 forward of an FP8 layer (moe_quant_forward_w8a8): dynamic 1x128
        FP8 activations on the FP8 matrix units."""
        return self._forward(logits, None, hidden, residual, out, workspace, probe, events,
                             stream, None, w8a8=True)

    def forward_w4a4(self, logits, hidden, act_gscale13: float, act_gscale2: float, residual=None,
                     out=None, workspace=None, probe: Optional[Dict] = None, events=None,
                     stream=None):
        """W4A4 forward of an NVFP4 layer (moe_quant_forward_w4a4): hidden rows
        and the SwiGLU intermediate quantized to NVFP4 with the calibrated
        global scales ``act_gscale13`` (gate/up input) and ``act_gscale2``
        (down input)."""
        return self._forward(logits, None, hidden, residual, out, workspace, probe, events,
                             stream, None, w4a4=(float(act_gscale13), float(act_gscale2)))

    def forward_with_router(self, router_w, hidden, residual=None, out=None, workspace=None,
                            logits_out=None, probe: Optional[Dict] = None, events=None,
                            stream=None):
        """Enqueue one forward whose router logits (BF16 gate ``router_w`` [E, H])
        are computed in the same kernel as the top-k; ``logits_out`` (float32
        [T, E]) optionally receives them."""
        return self._forward(None, router_w, hidden, residual, out, workspace, probe, events,
                             stream, logits_out)

    def forward_gated(self, gate: "Gate", hidden, logits=None, router_w=None, residual=None, out=None,
                      workspace=None, activations: str = "bf16", act_gscale13: float = 0.0,
                      act_gscale2: float = 0.0, logits_out=None, probe: Optional[Dict] = None,
                      events=None, stream=None):
        """Enqueue one forward under ``gate`` (moe_quant_forward_gated), from router
        ``logits`` or from the router weight ``router_w`` [E, H]; ``activations``:
        "bf16", "fp8" (FP8 layers) or "nvfp4" (NVFP4 layers, with the calibrated
        global scales)."""
        q = gate._q
        if (logits is None) == (router_w is None):
            raise ValueError("forward_gated needs exactly one of logits and router_w")
        if activations not in ACTIVATIONS:
            raise ValueError(f"unknown activations {activations!r}")
        if logits_out is not None and router_w is None:
            raise ValueError("logits_out needs router_w")
        if hidden.dim() != 2:
            raise ValueError("hidden must be [T, H]")
        index, t, bf16 = hidden.get_device(), hidden.shape[0], q.bf16
        if index >= 0 and index != q.device_now():
            with q.on(index):
                return self.forward_gated(gate, hidden, logits, router_w, residual, out, workspace, activations,
                                          act_gscale13, act_gscale2, logits_out, probe, events, stream)
        if gate.bias is not None and gate.bias.device != self.device:
            _on_gpu(self.device, **{"gate.bias": gate.bias})
        if out is None:
            out = _empty((t, self.hidden), bf16, self.device, stream)
        if workspace is None:
            workspace = _empty((max(self.workspace_size(t), 256),), q.u8, self.device, stream)
        shape, wide = (t, self.hidden), logits_out if logits is None else logits
        if (probe is None and events is None and index == self.device.index and t > 0
                and _fits(hidden, shape, bf16, index) and _fits(out, shape, bf16, index)
                and (residual is None or _fits(residual, shape, bf16, index))
                and (router_w is None or _fits(router_w, (self.num_experts, self.hidden), bf16, index))
                and (wide is None or _fits(wide, (t, self.num_experts), q.f32, index)
                     or (logits is not None and _fits(logits, (t, self.num_experts), bf16, index)))
                and workspace.is_contiguous() and workspace.get_device() == index
                and _nbytes(workspace) >= self._workspace_need(t)):
            # everything is as _forward's checks want it
            st = self._lib.moe_quant_forward_gated(
                self._h, gate._ref, _ptr(logits), MQ_BF16 if logits is not None and logits.dtype is bf16 else MQ_F32,
                _ptr(router_w), hidden.data_ptr(), _ptr(residual), t, out.data_ptr(), workspace.data_ptr(),
                _nbytes(workspace), ACTIVATIONS[activations], act_gscale13, act_gscale2, _ptr(logits_out), None,
                q.raw_stream(index) if stream is None else stream.cuda_stream)
            if st:
                _check(self._lib, st)
            return out
        return self._forward(logits, router_w, hidden, residual, out, workspace, probe, events, stream, logits_out,
                             gate=gate, act=(ACTIVATIONS[activations], float(act_gscale13), float(act_gscale2)))

    def _forward(self, logits, router_w, hidden, residual, out, workspace, probe, events, stream,
                 logits_out, w8a8=False, w4a4=None, gate=None, act=None):
        import torch
        if hidden.dim() != 2:
            raise ValueError("hidden must be [T, H]")
        t = hidden.shape[0]
        dev = self.device
        bf16 = (torch.bfloat16,)
        _need(hidden, "hidden", (t, self.hidden), bf16)
        if router_w is None:
            _need(logits, "logits", (t, self.num_experts), (torch.float32, torch.bfloat16))
        else:
            _need(router_w, "router_w", (self.num_experts, self.hidden), bf16)
            if logits_out is not None:
                _need(logits_out, "logits_out", (t, self.num_experts), (torch.float32,))
        if residual is not None:
            _need(residual, "residual", (t, self.hidden), bf16)
        if out is None:
            out = torch.empty((t, self.hidden), dtype=torch.bfloat16, device=dev)
        _need(out, "out", (t, self.hidden), bf16)
        shapes = {"topk_ids": ((t, self.top_k), torch.int32), "topk_w": ((t, self.top_k), torch.float32),
                  "expert_offsets": ((self.num_experts + 1,), torch.int32),
                  "sorted_token_ids": ((t * self.top_k,), torch.int32),
                  "inv_pos": ((t * self.top_k,), torch.int32),
                  "h": ((t * self.top_k, self.inter), torch.float16)}
        for name, v in (probe or {}).items():
            if name not in shapes:
                raise ValueError(f"unknown probe output {name!r}")
            if v is not None:
                _need(v, f"probe[{name!r}]", shapes[name][0], (shapes[name][1],))
        if workspace is not None and not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        _on_gpu(dev, hidden=hidden, logits=logits, router_w=router_w, residual=residual, out=out,
                workspace=workspace, logits_out=logits_out,
                **{f"probe[{n!r}]": v for n, v in (probe or {}).items()})
        if workspace is None:
            workspace = self.workspace(t, dev)
        if t > 0 and _nbytes(workspace) < self.workspace_size(t):   # T = 0 enqueues nothing
            raise ValueError(f"workspace holds {_nbytes(workspace)} bytes, "
                             f"{self.workspace_size(t)} needed for {t} tokens")
        pr = None
        if probe is not None or events is not None:
            pr = Probe()
            probe = probe or {}
            for name in ("topk_ids", "topk_w", "expert_offsets", "sorted_token_ids", "inv_pos", "h"):
                setattr(pr, name, _ptr(probe.get(name)))
            if events is not None:
                for i, ev in enumerate(events):
                    pr.events[i] = None if ev is None else ev.cuda_event
        prp = ctypes.byref(pr) if pr is not None else None
        if gate is not None:
            st = self._lib.moe_quant_forward_gated(
                self._h, gate._ref, _ptr(logits), MQ_F32 if logits is None else _mq_dtype(logits.dtype),
                _ptr(router_w), _ptr(hidden), _ptr(residual), t, _ptr(out), _ptr(workspace), _nbytes(workspace),
                *act, _ptr(logits_out), prp, _stream(stream))
        elif router_w is None:
            ldt = MQ_F32 if logits.dtype == torch.float32 else MQ_BF16
            if w4a4 is not None:
                st = self._lib.moe_quant_forward_w4a4(
                    self._h, _ptr(logits), ldt, _ptr(hidden), _ptr(residual), t, _ptr(out),
                    _ptr(workspace), _nbytes(workspace), w4a4[0], w4a4[1], prp, _stream(stream))
            else:
                fn = self._lib.moe_quant_forward_w8a8 if w8a8 else self._lib.moe_quant_forward
                st = fn(
                    self._h, _ptr(logits), ldt, _ptr(hidden), _ptr(residual), t, _ptr(out),
                    _ptr(workspace), _nbytes(workspace), prp, _stream(stream))
        else:
            st = self._lib.moe_quant_forward_with_router(
                self._h, _ptr(hidden), _ptr(router_w), _ptr(residual), t, _ptr(out),
                _ptr(workspace), _nbytes(workspace), _ptr(logits_out), prp, _stream(stream))
        _check(self._lib, st)
        return out

    def forward_noalloc(self, logits, hidden, residual=None, out=None, overflow_flag=None,
                        stream=None):
        """Enqueue one forward whose scratch is the library's static device
        array (moe_quant_forward_noalloc); ``overflow_flag``: None or an int32
        tensor of one element that receives the saturation flag."""
        import torch
        if hidden.dim() != 2:
            raise ValueError("hidden must be [T, H]")
        t = hidden.shape[0]
        dev = self.device
        bf16 = (torch.bfloat16,)
        _need(hidden, "hidden", (t, self.hidden), bf16)
        _need(logits, "logits", (t, self.num_experts), (torch.float32, torch.bfloat16))
        if residual is not None:
            _need(residual, "residual", (t, self.hidden), bf16)
        if out is None:
            out = torch.empty((t, self.hidden), dtype=torch.bfloat16, device=dev)
        _need(out, "out", (t, self.hidden), bf16)
        if overflow_flag is not None:
            _need(overflow_flag, "overflow_flag", (1,), (torch.int32,))
        _on_gpu(dev, hidden=hidden, logits=logits, residual=residual, out=out,
                overflow_flag=overflow_flag)
        ldt = MQ_F32 if logits.dtype == torch.float32 else MQ_BF16
        st = self._lib.moe_quant_forward_noalloc(
            self._h, _ptr(logits), ldt, _ptr(hidden), _ptr(residual), t, _ptr(out),
            _ptr(overflow_flag), _stream(stream))
        _check(self._lib, st)
        return out

    def check(self, workspace, stream=None) -> bool:
        """True if the last forward on ``workspace`` saturated its FP16 intermediate."""
        st = self._lib.moe_quant_check(self._h, _ptr(workspace), _stream(stream))
        if st == 9:
            return True
        _check(self._lib, st)
        return False

    def dequantize(self, which: int, expert: int, stream=None):
        import torch
        n, k = (2 * self.inter, self.hidden) if which == 0 else (self.hidden, self.inter)
        out = torch.empty((n, k), dtype=torch.float32, device=self.device)
        _check(self._lib, self._lib.moe_quant_dequantize(self._h, which, expert, _ptr(out),
                                                          _stream(stream)))
        return out

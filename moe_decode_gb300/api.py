"""Python binding of libmoe_decode.so (ctypes). Argument marshalling only:
every step of the layer runs in the library's CUDA kernels. Tensors are
torch CUDA tensors; their device pointers and the current stream are passed
through the C ABI declared in include/moe_decode.h.

There is no fallback: if the compiled library is missing, importing this
module raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_decode.so")

OK = 0
EINVAL, ESHAPE, EM, EWORKSPACE, EALIGN, ECUDA, ENODEVICE, ESCRATCH = -1, -2, -3, -4, -5, -6, -7, -8
EDEVICE_BAD_INDEX, ETIMEOUT, EDEVICE_OVERFLOW = -100, -101, -102
F_NO_PDL = 1
F_RESET_SCRATCH = 2
F_DEBUG_FORCE_TIMEOUT = 256
OPT_GRID_CTAS = 1
OPT_WAIT_TIMEOUT_NS = 2
OPT_TRACE_BUFFER = 3
OPT_DEBUG_HOLD_BACK = 4
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
LM_HEAD_WORKSPACE_BYTES = 1024
STATIC_SCRATCH_BYTES = 524288
PAGED_WORKSPACE_BYTES = 1024
PAGED_MAX_REQUESTS = 4096
TREE_MAX_TOKENS = 64
SAMPLE_MAX_VOCAB = 720896
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}
DTYPES = {torch.bfloat16: 0, torch.float16: 1}


class MoeError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {code} ({status_str(code)})")
        self.code = code


class Shape(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("inter", ctypes.c_int32), ("shared_inter", ctypes.c_int32), ("wfmt", ctypes.c_int32),
                ("scoring", ctypes.c_int32), ("routed_scale", ctypes.c_float), ("router_bias", ctypes.c_void_p),
                ("norm_weight", ctypes.c_void_p), ("norm_eps", ctypes.c_float), ("residual", ctypes.c_int32)]


class _Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w1", "w3", "w2", "s1", "s3", "s2", "ws1", "ws3", "ws2", "w2t",
                                                 "ws2t")]


class _KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + [
        (n, ctypes.c_int32) for n in ("dtype", "n_blocks", "block_size", "kv_heads", "head_dim")] + [
        (n, ctypes.c_int64) for n in ("k_block_stride", "k_token_stride", "k_head_stride", "v_block_stride",
                                      "v_token_stride", "v_head_stride")]


class _KvCache8(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] + [
        (n, ctypes.c_int32) for n in ("n_blocks", "block_size", "kv_heads", "head_dim")] + [
        (n, ctypes.c_int64) for n in ("k_block_stride", "k_token_stride", "k_head_stride", "v_block_stride",
                                      "v_token_stride", "v_head_stride")]


class _RopeAngles(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("scale", ctypes.c_float)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m moe_decode_gb300.build` "
                          "(there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    sp = ctypes.POINTER(Shape)
    wp = ctypes.POINTER(_Weights)
    lib.moe_workspace_bytes.argtypes = [sp, I32]
    lib.moe_workspace_bytes.restype = SZ
    lib.moe_workspace_init.argtypes = [P, SZ, P]
    lib.moe_route.argtypes = [P, I32, P, sp, P, P, P, SZ, P]
    lib.moe_ffn.argtypes = [P, I32, P, P, wp, sp, P, P, SZ, P]
    lib.moe_decode_layer.argtypes = [P, I32, P, wp, sp, P, P, P, P, SZ, ctypes.c_uint32, P]
    lib.moe_decode_layer_static_scratch.argtypes = [P, I32, P, wp, sp, P, P, P, ctypes.c_uint32, P]
    lib.moe_read_status.argtypes = [P, P, ctypes.POINTER(ctypes.c_int32)]
    lib.moe_static_scratch_status.argtypes = [P, ctypes.POINTER(ctypes.c_int32)]
    lib.moe_status_str.argtypes = [I32]
    lib.moe_status_str.restype = ctypes.c_char_p
    lib.moe_mxfp4_dequant.argtypes = [P, P, I64, I32, P, P]
    lib.moe_set_option.argtypes = [I32, I64]
    lib.moe_lm_head.argtypes = [P, I32, P, P, I32, I32, I32, P, P, SZ, ctypes.c_uint32, P]
    lib.moe_fp8_quantize.argtypes = [P, I64, I32, I32, P, P, P]
    lib.moe_fp8_dequant.argtypes = [P, P, I64, I32, I32, P, P]
    lib.moe_transpose_down.argtypes = [P, I64, I32, I32, P, P]
    F32, cp = ctypes.c_float, ctypes.POINTER(_KvCache)
    lib.moe_paged_plan.argtypes = [P, P, I32, P, I32, P, P, I32, I32, P, P, P, P, I32, P, P, SZ, P]
    lib.moe_paged_append.argtypes = [P, I64, I64, P, I64, I64, I32, P, cp, P, SZ, P]
    lib.moe_paged_attention_workspace_bytes.argtypes = [I32, cp]
    lib.moe_paged_attention_workspace_bytes.restype = SZ
    lib.moe_paged_attention.argtypes = [P, I64, I64, I32, I32, cp, P, I32, P, P, I32, F32, I32, P, P, P, SZ, P]
    lib.moe_sample.argtypes = [P, I32, I32, I32, I64, P, P, P, P, P, P, P, P]
    F64, rp, c8 = ctypes.c_double, ctypes.POINTER(_RopeAngles), ctypes.POINTER(_KvCache8)
    lib.moe_rope_table.argtypes = [I32, F64, I32, F64, I32, F64, F64, P, ctypes.POINTER(F32)]
    lib.moe_rope_turns.argtypes = [P, I32, P]
    rows = [P, I64, I64]
    lib.moe_rope.argtypes = [*rows, *rows, I32, *rows, *rows, I32, I32, I32, I32, P, rp, P]
    lib.moe_paged_rope_append.argtypes = [*rows, *rows, I32, *rows, *rows, I32, P, P, rp, cp, P, SZ, P]
    lib.moe_paged_rope_append8.argtypes = [*rows, *rows, I32, *rows, *rows, I32, I32, P, P, rp, c8, P, SZ, P]
    lib.moe_paged_append8.argtypes = [*rows, *rows, I32, I32, P, c8, P, SZ, P]
    lib.moe_tree_plan.argtypes = [P, P, P, I32, I32, P, P, P, SZ, P]
    lib.moe_paged_tree_attention.argtypes = [P, I64, I64, I32, I32, cp, P, I32, P, P, P, I32, F32, P, P, P, SZ, P]
    lib.moe_paged_attention8_workspace_bytes.argtypes = [I32, c8]
    lib.moe_paged_attention8_workspace_bytes.restype = SZ
    lib.moe_paged_attention8.argtypes = [P, I64, I64, I32, I32, I32, c8, P, I32, P, P, P, I32, F32, I32, P, P, P, SZ, P]
    lib.moe_paged_read.argtypes = [cp, P, I32, *rows, *rows, P, SZ, P]
    lib.moe_paged_read8.argtypes = [c8, P, I32, I32, *rows, *rows, P, SZ, P]
    lib.moe_last_launch_count.argtypes = []
    for f in ("moe_workspace_init", "moe_route", "moe_ffn", "moe_decode_layer", "moe_decode_layer_static_scratch",
              "moe_read_status", "moe_static_scratch_status", "moe_mxfp4_dequant", "moe_set_option", "moe_last_launch_count",
              "moe_lm_head", "moe_fp8_quantize", "moe_fp8_dequant", "moe_transpose_down",
              "moe_paged_plan", "moe_paged_append", "moe_paged_attention", "moe_sample", "moe_rope_table", "moe_rope_turns",
              "moe_rope", "moe_paged_rope_append", "moe_paged_rope_append8", "moe_paged_append8", "moe_paged_read",
              "moe_paged_read8", "moe_tree_plan", "moe_paged_tree_attention", "moe_paged_attention8"):
        getattr(lib, f).restype = I32
    return lib


lib = _load()


def status_str(code: int) -> str:
    return lib.moe_status_str(code).decode()


def _check(rc: int, what: str):
    if rc != OK:
        raise MoeError(rc, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def make_shape(hidden, n_experts, top_k, inter, shared_inter, wfmt=0, scoring: int = 0, routed_scale: float = 0.0,
               router_bias: Optional[torch.Tensor] = None, norm_weight: Optional[torch.Tensor] = None,
               norm_eps: float = 0.0, residual: bool = False) -> Shape:
    """Layer shape, router configuration and input/output options;
    router_bias (fp32 [E]) and norm_weight (bf16 [H]) are device tensors that
    must stay alive while the shape is used."""
    return Shape(hidden, n_experts, top_k, inter, shared_inter, wfmt, scoring, routed_scale,
                 None if router_bias is None else router_bias.data_ptr(),
                 None if norm_weight is None else norm_weight.data_ptr(), norm_eps, int(residual))


@dataclass
class ExpertWeights:
    """Device tensors of one layer's experts (layouts in include/moe_decode.h).
    bf16: w1, w3 [E,I,H], w2 [E,H,I]; MXFP4: w1, w3 u8 [E,I,H/2], s1, s3 u8
    [E,I,H/32], w2 u8 [E,H,I/2], s2 u8 [E,H,I/32]; FP8: w1, w3 u8 [E,I,H],
    s1, s3 fp32 [E,I,H/128], w2 u8 [E,H,I], s2 fp32 [E,H,I/128]. Shared
    expert bf16."""
    w1: torch.Tensor
    w3: torch.Tensor
    w2: torch.Tensor
    ws1: Optional[torch.Tensor] = None
    ws3: Optional[torch.Tensor] = None
    ws2: Optional[torch.Tensor] = None
    s1: Optional[torch.Tensor] = None
    s3: Optional[torch.Tensor] = None
    s2: Optional[torch.Tensor] = None
    w2t: Optional[torch.Tensor] = None   # bf16 [E, I, H] (transpose_down(w2)); one-token split-K layer
    ws2t: Optional[torch.Tensor] = None  # bf16 [Is, H]

    def cstruct(self) -> _Weights:
        return _Weights(*(None if t is None else t.data_ptr() for t in
                          (self.w1, self.w3, self.w2, self.s1, self.s3, self.s2, self.ws1, self.ws3, self.ws2,
                           self.w2t, self.ws2t)))


def workspace_bytes(shape: Shape, M: int) -> int:
    return int(lib.moe_workspace_bytes(ctypes.byref(shape), M))


def workspace_init(ws: torch.Tensor, stream=None):
    _check(lib.moe_workspace_init(_ptr(ws), ws.numel(), _stream(stream)), "moe_workspace_init")


def workspace(shape: Shape, M: int, device="cuda", stream=None) -> torch.Tensor:
    n = workspace_bytes(shape, M)
    if n == 0:
        raise MoeError(ESHAPE, "moe_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    workspace_init(ws, stream)
    return ws


def route(x, Wg, shape: Shape, idx, w, ws, stream=None):
    _check(lib.moe_route(_ptr(x), x.shape[0], _ptr(Wg), ctypes.byref(shape), _ptr(idx), _ptr(w), _ptr(ws),
                         ws.numel(), _stream(stream)), "moe_route")


def ffn(x, idx, w, weights: ExpertWeights, shape: Shape, y, ws, stream=None):
    cw = weights.cstruct()
    _check(lib.moe_ffn(_ptr(x), x.shape[0], _ptr(idx), _ptr(w), ctypes.byref(cw), ctypes.byref(shape), _ptr(y),
                       _ptr(ws), ws.numel(), _stream(stream)), "moe_ffn")


def decode_layer(x, Wg, weights: ExpertWeights, shape: Shape, y, ws, idx_out=None, w_out=None, flags: int = 0,
                 stream=None, cweights: Optional[_Weights] = None):
    cw = cweights if cweights is not None else weights.cstruct()
    _check(lib.moe_decode_layer(_ptr(x), x.shape[0], _ptr(Wg), ctypes.byref(cw), ctypes.byref(shape),
                                _ptr(idx_out), _ptr(w_out), _ptr(y), _ptr(ws), ws.numel(), flags,
                                _stream(stream)), "moe_decode_layer")


def decode_layer_static_scratch(x, Wg, weights: ExpertWeights, shape: Shape, y, idx_out=None, w_out=None,
                                flags: int = 0, stream=None, cweights: Optional[_Weights] = None):
    cw = cweights if cweights is not None else weights.cstruct()
    _check(lib.moe_decode_layer_static_scratch(_ptr(x), x.shape[0], _ptr(Wg), ctypes.byref(cw),
                                               ctypes.byref(shape), _ptr(idx_out), _ptr(w_out), _ptr(y), flags,
                                               _stream(stream)), "moe_decode_layer_static_scratch")


def read_status(ws, stream=None) -> int:
    v = ctypes.c_int32(0)
    _check(lib.moe_read_status(_ptr(ws), _stream(stream), ctypes.byref(v)), "moe_read_status")
    return v.value


def static_scratch_status(stream=None) -> int:
    """Device status word of this device's static scratch (synchronises)."""
    v = ctypes.c_int32(0)
    _check(lib.moe_static_scratch_status(_stream(stream), ctypes.byref(v)), "moe_static_scratch_status")
    return v.value


def mxfp4_dequant(codes, scales, K: int, out, stream=None):
    rows = codes.numel() // (K // 2)
    _check(lib.moe_mxfp4_dequant(_ptr(codes), _ptr(scales), rows, K, _ptr(out), _stream(stream)),
           "moe_mxfp4_dequant")


def set_option(option: int, value: int):
    _check(lib.moe_set_option(option, value), "moe_set_option")


def last_launch_count() -> int:
    return int(lib.moe_last_launch_count())


def lm_head(x, W, V: int, H: int, logits, ws, wfmt: int = 0, w_scale=None, flags: int = 0, stream=None):
    """logits fp32 [M, V] = x bf16 [M, H] . W^T; W bf16 [V, H] (wfmt 0) or e4m3
    codes u8 [V, H] with fp32 per-row scales w_scale [V] (wfmt 2)."""
    _check(lib.moe_lm_head(_ptr(x), x.shape[0], _ptr(W), _ptr(w_scale), V, H, wfmt, _ptr(logits), _ptr(ws),
                           ws.numel(), flags, _stream(stream)), "moe_lm_head")


def fp8_quantize(w, block: int, codes, scales, stream=None):
    rows, K = w.shape
    _check(lib.moe_fp8_quantize(_ptr(w), rows, K, block, _ptr(codes), _ptr(scales), _stream(stream)),
           "moe_fp8_quantize")


def transpose_down(w2: torch.Tensor, stream=None) -> torch.Tensor:
    """Transposed copy of down projections (moe_transpose_down): bf16
    [n, H, I] (or [H, I]) -> [n, I, H] (or [I, H]), for the split-K one-token
    layer. Weight preparation, not the hot path."""
    src = w2 if w2.dim() == 3 else w2.unsqueeze(0)
    n, H, I = src.shape
    out = torch.empty((n, I, H), dtype=w2.dtype, device=w2.device)
    _check(lib.moe_transpose_down(_ptr(src), n, H, I, _ptr(out), _stream(stream)), "moe_transpose_down")
    return out if w2.dim() == 3 else out[0]


def fp8_dequant(codes, scales, block: int, out, stream=None):
    rows, K = codes.shape
    _check(lib.moe_fp8_dequant(_ptr(codes), _ptr(scales), rows, K, block, _ptr(out), _stream(stream)),
           "moe_fp8_dequant")


# ---------------------------------------------------------------- paged step
def _want(ok: bool, what: str, code: int = EINVAL):
    if not ok:
        raise MoeError(code, what)


_INT32 = 1 << 31


def _int32(what: str, n: int):
    """A whole number that the library takes in 32 bits (ctypes drops what is above)."""
    if not -_INT32 <= n < _INT32:
        raise MoeError(ESHAPE, f"{what} beyond 32 bits")


def _raw(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


# The current stream's handle without a Stream object around it: 0.3 us a
# call where torch.cuda.current_stream() takes 2.9 (measured on the host of a
# GB300), of a call whose launch takes 4. Alike the current device: where a
# tensor is on one, torch.cuda is initialised.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _raw_stream(stream, dev: int) -> int:
    if stream is not None:
        if stream.device_index != dev:
            raise MoeError(EINVAL, f"a stream of device {stream.device_index}, the current device is {dev}")
        return stream.cuda_stream
    if _current_raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _current_raw_stream(dev)


def _device(what: str, t: torch.Tensor) -> int:
    """The current device, where a call launches: every tensor of the call has
    to be there (get_device() is -1 for host memory)."""
    if not t.is_cuda:
        raise MoeError(EINVAL, f"{what}: tensors on the device, got {t.device}")
    return _current_device()


def _workspace(what: str, dev: int, ws: torch.Tensor):
    if ws.dtype is not torch.uint8 or ws.get_device() != dev or not ws.is_contiguous():
        raise MoeError(EINVAL, f"{what}: ws uint8, contiguous, on the current device (paged_workspace); got {ws.dtype} on {ws.device}")


def _vectors(what: str, dev: int, dtype: torch.dtype, *pairs):
    """Each pair (tensor or None, elements or None for any number): contiguous
    tensors of one dtype on the current device."""
    for t, n in pairs:
        if t is not None and (t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous()
                              or (n is not None and t.numel() != n)):
            raise MoeError(EINVAL, f"{what}: {dtype}, contiguous, on the current device, "
                                   f"{n if n is not None else 'any number of'} elements; got {t.dtype} {tuple(t.shape)} on {t.device}")


class KvCache:
    """A paged KV cache: K and V [n_blocks, block_size, kv_heads, head_dim]
    bf16 or fp16 views (any strides that are multiples of 8 elements, the last
    dimension contiguous: `.transpose(1, 2)` of a [block, head, token, d]
    buffer is one), on the device of the calls that use it. Keeps the tensors
    alive; build it once, next to them."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        _want(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype and k.dtype in DTYPES
              and k.stride(3) == 1 and v.stride(3) == 1, "KvCache: K and V [blocks, tokens, heads, d], one dtype", ESHAPE)
        _want(k.get_device() == v.get_device(), "KvCache: K and V on one device")
        self.k, self.v = k, v
        self.device_index = k.get_device()
        n_blocks, self.block_size, self.kv_heads, self.head_dim = k.shape
        # (a dimension of one element has no stride of its own: what a view says
        # there may be anything)
        sk, sv = ([t.stride(i) if t.shape[i] > 1 else (self.head_dim + 7) // 8 * 8 for i in range(3)] for t in (k, v))
        self.dtype = k.dtype
        self._c = _KvCache(k.data_ptr(), v.data_ptr(), DTYPES[k.dtype], n_blocks, self.block_size, self.kv_heads,
                           self.head_dim, sk[0], sk[1], sk[2], sv[0], sv[1], sv[2])
        self._ref = ctypes.pointer(self._c)


class KvCache8:
    """A paged KV cache of e4m3 codes with one power of two for each token and
    head (moe_kv_cache8): K and V [n_blocks, block_size, kv_heads, head_dim]
    uint8 or float8_e4m3fn views (strides multiples of 16, the last dimension
    contiguous), k_scale and v_scale uint8 [n_blocks, kv_heads, block_size]
    contiguous (e8m0: 2^(byte - 127), 255 for NaN). KvCache8.empty makes one.
    Takes the place of a KvCache in paged_append, paged_rope_append,
    paged_attention and paged_read; their other tensors are bf16 or fp16."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        _want(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype and k.dtype in (torch.uint8, torch.float8_e4m3fn)
              and k.stride(3) == 1 and v.stride(3) == 1, "KvCache8: K and V [blocks, tokens, heads, d], uint8 or float8_e4m3fn", ESHAPE)
        n_blocks, self.block_size, self.kv_heads, self.head_dim = k.shape
        for s in (k_scale, v_scale):
            _want(s.dtype is torch.uint8 and s.shape == (n_blocks, self.kv_heads, self.block_size) and s.is_contiguous(),
                  "KvCache8: k_scale and v_scale uint8 [blocks, heads, tokens], contiguous", ESHAPE)
        _want(k.get_device() == v.get_device() == k_scale.get_device() == v_scale.get_device(), "KvCache8: all tensors on one device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device_index = k.get_device()
        # (a dimension of one element has no stride of its own)
        sk, sv = ([t.stride(i) if t.shape[i] > 1 else (self.head_dim + 15) // 16 * 16 for i in range(3)] for t in (k, v))
        self._c = _KvCache8(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), n_blocks, self.block_size,
                            self.kv_heads, self.head_dim, *sk, *sv)
        self._ref = ctypes.pointer(self._c)

    @classmethod
    def empty(cls, n_blocks: int, block_size: int, kv_heads: int, head_dim: int, device="cuda") -> "KvCache8":
        k, v = (torch.zeros((n_blocks, block_size, kv_heads, head_dim), dtype=torch.uint8, device=device) for _ in range(2))
        ks, vs = (torch.zeros((n_blocks, kv_heads, block_size), dtype=torch.uint8, device=device) for _ in range(2))
        return cls(k, v, ks, vs)


def paged_workspace(q_heads: int = 0, cache: "Optional[KvCache | KvCache8]" = None, device="cuda", stream=None) -> torch.Tensor:
    """A zeroed workspace for the paged-step calls: for paged_attention with
    q_heads over `cache`, or, without them, for the other calls. One for the
    largest serves them all, one call after another."""
    need = lib.moe_paged_attention8_workspace_bytes if isinstance(cache, KvCache8) else lib.moe_paged_attention_workspace_bytes
    n = PAGED_WORKSPACE_BYTES if cache is None else int(need(q_heads, cache._ref))
    _want(n > 0, "moe_paged_attention_workspace_bytes", ESHAPE)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    workspace_init(ws, stream)
    return ws


def paged_plan(ctx_lens, new_lens, free_list, block_tables, block_size: int, q_start, seq_lens, slot_map, taken, ws,
               positions=None, free_head=None, stream=None):
    """Block tables and slot map of a step (moe_paged_plan). All int32 device
    tensors: ctx_lens, new_lens [B], free_list [F], block_tables [B, W]
    (updated in place), outputs q_start [B + 1], seq_lens [B], slot_map [T],
    positions [T], taken [1]; free_head [1] is where the free list begins."""
    B, T = ctx_lens.numel(), slot_map.numel()
    _want(block_tables.dim() == 2 and block_tables.shape[0] == B, "paged_plan: block_tables int32 [B, W]")
    _int32("paged_plan: block_size", block_size)
    dev = _device("paged_plan", ctx_lens)
    _vectors("paged_plan", dev, torch.int32, (ctx_lens, B), (new_lens, B), (free_list, None), (free_head, 1),
             (block_tables, None), (q_start, B + 1), (seq_lens, B), (slot_map, T), (positions, T), (taken, 1))
    _workspace("paged_plan", dev, ws)
    rc = lib.moe_paged_plan(ctx_lens.data_ptr(), new_lens.data_ptr(), B, free_list.data_ptr(), free_list.numel(),
                            _raw(free_head), block_tables.data_ptr(), block_tables.shape[1], block_size,
                            q_start.data_ptr(), seq_lens.data_ptr(), slot_map.data_ptr(), _raw(positions), T,
                            taken.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(stream, dev))
    if rc:
        raise MoeError(rc, "moe_paged_plan")


def tree_plan(parents, q_start, seq_lens, masks, positions, ws, stream=None):
    """Masks int64 [T] and positions int32 [T] (or None) of trees of drafted
    tokens from parents int32 [T] (moe_tree_plan): each token's parent among its
    request's new tokens, -1 for the token before them; q_start int32 [B + 1],
    seq_lens int32 [B] as paged_plan gives them."""
    T, B = parents.numel(), seq_lens.numel()
    dev = _device("tree_plan", parents)
    _vectors("tree_plan: parents, q_start, seq_lens, positions", dev, torch.int32, (parents, T), (q_start, B + 1), (seq_lens, B), (positions, T))
    _vectors("tree_plan: masks", dev, torch.int64, (masks, T))
    _workspace("tree_plan", dev, ws)
    rc = lib.moe_tree_plan(parents.data_ptr(), q_start.data_ptr(), seq_lens.data_ptr(), B, T, masks.data_ptr(), _raw(positions),
                           ws.data_ptr(), ws.numel(), _raw_stream(stream, dev))
    if rc:
        raise MoeError(rc, "moe_tree_plan")


def _rows(what: str, dev: int, dtype: torch.dtype, shape, t: torch.Tensor, out: bool = False):
    """(address, token stride, head stride) of [T, heads, d] on the current
    device. A dimension of one element has no stride of its own: 0, or of an
    output one that its rows would have."""
    strides = t.stride()
    if t.shape != shape:
        raise MoeError(ESHAPE, f"{what}: {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype or t.get_device() != dev or strides[2] != 1:
        raise MoeError(EINVAL, f"{what}: {dtype}, the last dimension contiguous, on the current device; got {t.dtype} on {t.device}")
    token, head = strides[0], strides[1]
    if shape[1] == 1:
        head = (shape[2] + 7) // 8 * 8 if out else 0
    if shape[0] == 1:
        token = (shape[2] + 7) // 8 * 8 * shape[1] if out else 0
    return t.data_ptr(), token, head


def _pair(what: str, dev: int, dtype: torch.dtype, shape, t: torch.Tensor, out: Optional[torch.Tensor]):
    """_rows of an input and of its output, which is the input's place without one."""
    o = _rows(what, dev, dtype, shape, t if out is None else out, True)
    if out is None or out is t:
        return (*o, *o)
    i = _rows(what, dev, dtype, shape, t)
    return (*(o if i[0] == o[0] and (shape[0] == 1 or i[1] == o[1]) and (shape[1] == 1 or i[2] == o[2]) else i), *o)


_NO_PAIR = (None, 0, 0, None, 0, 0)


def paged_append(k_new, v_new, slot_map, cache, ws, stream=None):
    """Writes k_new, v_new [T, kv_heads, head_dim] (last dimension contiguous,
    e.g. slices of a fused projection's output) to the cache's slots
    slot_map [T] (moe_paged_append, or moe_paged_append8 into a KvCache8)."""
    T = k_new.shape[0]
    _want(k_new.shape == (T, cache.kv_heads, cache.head_dim) and v_new.shape == k_new.shape,
          "paged_append: k_new, v_new [T, kv_heads, head_dim]", ESHAPE)
    dev = _device("paged_append", k_new)
    codes = isinstance(cache, KvCache8)
    dtype = k_new.dtype if codes and k_new.dtype in DTYPES else torch.bfloat16 if codes else cache.dtype
    _want(k_new.dtype == dtype and v_new.dtype == dtype and k_new.stride(2) == 1 and v_new.stride(2) == 1
          and k_new.get_device() == v_new.get_device() == cache.device_index == dev,
          "paged_append: k_new, v_new of the cache's dtype (KvCache8: bf16 or fp16), all on the current device")
    _vectors("paged_append: slot_map", dev, torch.int32, (slot_map, T))
    _workspace("paged_append", dev, ws)
    kt, kh, _ = k_new.stride()
    vt, vh, _ = v_new.stride()
    if T == 1:
        kt = vt = 0
    if cache.kv_heads == 1:
        kh = vh = 0
    if codes:
        rc = lib.moe_paged_append8(k_new.data_ptr(), kt, kh, v_new.data_ptr(), vt, vh, T, DTYPES[dtype], slot_map.data_ptr(),
                                   cache._ref, ws.data_ptr(), ws.numel(), _raw_stream(stream, dev))
    else:
        rc = lib.moe_paged_append(k_new.data_ptr(), kt, kh, v_new.data_ptr(), vt, vh, T, slot_map.data_ptr(), cache._ref,
                                  ws.data_ptr(), ws.numel(), _raw_stream(stream, dev))
    if rc:
        raise MoeError(rc, "moe_paged_append8" if codes else "moe_paged_append")


class Rope:
    """Angles of rotary positions (moe_rope_angles): how fast each pair of the
    first rotary_dim dimensions turns, as integers on the device. scaling:
    "none", "linear", "ntk", "yarn" or "bands" for contexts `factor` times the
    `context` a model was made for (moe_rope_table; low and high are the
    borders in turns, 0 for the usual ones); scale: of the rotated values, None
    for the scaling's own. Rope.of(frequencies) takes any frequencies."""

    def __init__(self, rotary_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
                 factor: float = 1.0, context: int = 0, low: float = 0.0, high: float = 0.0, scale: Optional[float] = None,
                 device="cuda"):
        _want(scaling in ROPE_SCALINGS, f"Rope: scaling one of {', '.join(ROPE_SCALINGS)}")
        _want(0 < rotary_dim <= 512, "Rope: rotary_dim", ESHAPE)
        _int32("Rope: context", context)
        turns = (ctypes.c_uint64 * max(1, rotary_dim // 2))()
        own = ctypes.c_float(1.0)
        _check(lib.moe_rope_table(rotary_dim, base, ROPE_SCALINGS[scaling], factor, context, low, high, turns,
                                  ctypes.byref(own)), "moe_rope_table")
        self._set(turns, rotary_dim, interleaved, own.value if scale is None else scale, device)

    @classmethod
    def of(cls, frequencies, interleaved: bool = False, scale: float = 1.0, device="cuda") -> "Rope":
        """frequencies: radians a position of each pair (numbers of 64 bits)."""
        f = [float(x) for x in frequencies]
        turns = (ctypes.c_uint64 * max(1, len(f)))()
        _check(lib.moe_rope_turns((ctypes.c_double * max(1, len(f)))(*f), len(f), turns), "moe_rope_turns")
        self = cls.__new__(cls)
        self._set(turns, 2 * len(f), interleaved, scale, device)
        return self

    def _set(self, turns, rotary_dim, interleaved, scale, device):
        # (the same 64 bits in torch's signed integers)
        signed = [t - (1 << 64) if t >= 1 << 63 else t for t in turns]
        self.turns = torch.tensor(signed, dtype=torch.int64, device=device)
        self.rotary_dim, self.interleaved, self.scale = rotary_dim, bool(interleaved), scale
        self.device_index = self.turns.get_device()
        self._c = _RopeAngles(self.turns.data_ptr(), rotary_dim, int(interleaved), scale)
        self._ref = ctypes.pointer(self._c)


def rope(q, k, positions, angles: Rope, q_out=None, k_out=None, stream=None):
    """Rotates q [T, q_heads, head_dim] and k [T, kv_heads, head_dim] (or
    None) to the positions int32 [T] (moe_rope): into q_out and k_out, or in
    place. bf16 or fp16, the last dimension contiguous; rows at a negative
    position stay as they are."""
    T, heads, d = q.shape
    dev = _device("rope", q)
    dtype = q.dtype
    _want(dtype in DTYPES, "rope: q bf16 or fp16")
    qs = _pair("rope: q, q_out", dev, dtype, q.shape, q, q_out)
    kv, ks = 0, _NO_PAIR
    if k is not None:
        kv = k.shape[1]
        ks = _pair("rope: k, k_out", dev, dtype, (T, kv, d), k, k_out)
    else:
        _want(k_out is None, "rope: k_out without k")
    _vectors("rope: positions", dev, torch.int32, (positions, T))
    _want(angles.device_index == dev, "rope: angles on the current device")
    rc = lib.moe_rope(*qs, heads, *ks, kv, T, d, DTYPES[dtype], positions.data_ptr(), angles._ref, _raw_stream(stream, dev))
    if rc:
        raise MoeError(rc, "moe_rope")


def paged_rope_append(q, k_new, v_new, positions, slot_map, angles: Rope, cache, ws, q_out=None, stream=None):
    """rope and paged_append in one launch (moe_paged_rope_append, or
    moe_paged_rope_append8 into a KvCache8): q [T, q_heads, head_dim] (or None)
    rotated into q_out or in place, k_new [T, kv_heads, head_dim] rotated and
    v_new as it is into the cache's slots slot_map [T]; k_new keeps its values."""
    T = k_new.shape[0]
    d = cache.head_dim
    dev = _device("paged_rope_append", k_new)
    codes = isinstance(cache, KvCache8)
    dtype = k_new.dtype if codes else cache.dtype
    _want(dtype in DTYPES and cache.device_index == dev and angles.device_index == dev,
          "paged_rope_append: bf16 or fp16, cache and angles on the current device")
    ks = _rows("paged_rope_append: k_new, v_new", dev, dtype, (T, cache.kv_heads, d), k_new)
    vs = _rows("paged_rope_append: k_new, v_new", dev, dtype, (T, cache.kv_heads, d), v_new)
    heads, qs = 0, _NO_PAIR
    if q is not None:
        heads = q.shape[1]
        qs = _pair("paged_rope_append: q, q_out", dev, dtype, (T, heads, d), q, q_out)
    else:
        _want(q_out is None, "paged_rope_append: q_out without q")
    _vectors("paged_rope_append: positions, slot_map", dev, torch.int32, (positions, T), (slot_map, T))
    _workspace("paged_rope_append", dev, ws)
    args = (*qs, heads, *ks, *vs, T)
    rest = (positions.data_ptr(), slot_map.data_ptr(), angles._ref, cache._ref, ws.data_ptr(), ws.numel(), _raw_stream(stream, dev))
    rc = lib.moe_paged_rope_append8(*args, DTYPES[dtype], *rest) if codes else lib.moe_paged_rope_append(*args, *rest)
    if rc:
        raise MoeError(rc, "moe_paged_rope_append8" if codes else "moe_paged_rope_append")


def paged_read(cache, slot_map, k_out, v_out, ws, stream=None):
    """Reads the slots slot_map [T] back into k_out, v_out [T, kv_heads,
    head_dim] (moe_paged_read, of the cache's dtype, or moe_paged_read8 of a
    KvCache8, bf16 or fp16); rows of slot -1 stay as they are."""
    T = slot_map.numel()
    dev = _device("paged_read", slot_map)
    codes = isinstance(cache, KvCache8)
    dtype = k_out.dtype if codes else cache.dtype
    _want(dtype in DTYPES and cache.device_index == dev, "paged_read: bf16 or fp16, cache on the current device")
    shape = (T, cache.kv_heads, cache.head_dim)
    ks, vs = (_rows("paged_read: k_out, v_out", dev, dtype, shape, t, True) for t in (k_out, v_out))
    _vectors("paged_read: slot_map", dev, torch.int32, (slot_map, T))
    _workspace("paged_read", dev, ws)
    out = (*ks, *vs, ws.data_ptr(), ws.numel(), _raw_stream(stream, dev))
    if codes:
        rc = lib.moe_paged_read8(cache._ref, slot_map.data_ptr(), T, DTYPES[dtype], *out)
    else:
        rc = lib.moe_paged_read(cache._ref, slot_map.data_ptr(), T, *out)
    if rc:
        raise MoeError(rc, "moe_paged_read8" if codes else "moe_paged_read")


def paged_attention(q, cache, block_tables, q_start, seq_lens, out, ws, lse=None, scale: float = 0.0,
                    window: int = 0, stream=None, tree_masks=None):
    """Attention of the step's tokens q [T, q_heads, head_dim] over the paged
    cache (moe_paged_attention; moe_paged_attention8 over a KvCache8, of bf16 or
    fp16 queries): out [T, q_heads, head_dim] contiguous, lse fp32 [T, q_heads]
    or None; block_tables int32 [B, W], q_start int32 [B + 1], seq_lens int32
    [B] as paged_plan gives them; window > 0: only the last `window` keys;
    scale <= 0: 1 / sqrt(head_dim). tree_masks int64 [T] from tree_plan: of its
    request's new tokens a row sees those that its mask names
    (moe_paged_tree_attention; without a window)."""
    T, heads, d = q.shape
    B = seq_lens.numel()
    codes = isinstance(cache, KvCache8)
    dtype = q.dtype if codes else cache.dtype
    _want(d == cache.head_dim and out.shape == q.shape, "paged_attention: q, out [T, q_heads, head_dim]", ESHAPE)
    dev = _device("paged_attention", q)
    _want(q.dtype == dtype and dtype in DTYPES and out.dtype == dtype and q.stride(2) == 1 and out.is_contiguous()
          and q.get_device() == out.get_device() == cache.device_index == dev,
          "paged_attention: q, out of the cache's dtype (KvCache8: bf16 or fp16), all on the current device")
    _want(block_tables.dim() == 2 and block_tables.shape[0] == B, "paged_attention: block_tables int32 [B, W]")
    _vectors("paged_attention: block_tables, q_start, seq_lens", dev, torch.int32, (block_tables, None), (q_start, B + 1),
             (seq_lens, B))
    _vectors("paged_attention: lse", dev, torch.float32, (lse, T * heads))
    _vectors("paged_attention: tree_masks", dev, torch.int64, (tree_masks, T))
    _want(tree_masks is None or window == 0, "paged_attention: tree_masks and a window", ESHAPE)
    _int32("paged_attention: window", window)
    _workspace("paged_attention", dev, ws)
    qt, qh, _ = q.stride()
    if T == 1:
        qt = 0
    if heads == 1:
        qh = 0
    queries = (q.data_ptr(), qt, qh, T, heads)
    step = (cache._ref, block_tables.data_ptr(), block_tables.shape[1], q_start.data_ptr(), seq_lens.data_ptr())
    rest = (out.data_ptr(), _raw(lse), ws.data_ptr(), ws.numel(), _raw_stream(stream, dev))
    if codes:
        name = "moe_paged_attention8"
        rc = lib.moe_paged_attention8(*queries, DTYPES[dtype], *step, _raw(tree_masks), B, scale, window, *rest)
    elif tree_masks is not None:
        name = "moe_paged_tree_attention"
        rc = lib.moe_paged_tree_attention(*queries, *step, tree_masks.data_ptr(), B, scale, *rest)
    else:
        name = "moe_paged_attention"
        rc = lib.moe_paged_attention(*queries, *step, B, scale, window, *rest)
    if rc:
        raise MoeError(rc, name)


_LOGITS = {torch.float32: 0, torch.bfloat16: 1}


def sample(logits, u, tokens, probs=None, temperature=None, top_k=None, top_p=None, min_p=None, stream=None):
    """One token from each row of logits [M, V] (fp32 or bf16) with the random
    numbers u fp32 [M] in [0, 1) (moe_sample): tokens int32 [M], probs fp32
    [M] or None; per-row settings temperature, top_p, min_p fp32 [M], top_k
    int32 [M], None for off."""
    M, V = logits.shape
    dev = _device("sample", logits)
    _want(logits.dtype in _LOGITS and logits.get_device() == dev and (V == 1 or logits.stride(1) == 1),
          "sample: logits fp32 or bf16 [M, V], rows contiguous, on the current device")
    _vectors("sample: u, probs, temperature, top_p, min_p", dev, torch.float32, (u, M), (probs, M), (temperature, M),
             (top_p, M), (min_p, M))
    _vectors("sample: tokens, top_k", dev, torch.int32, (tokens, M), (top_k, M))
    rc = lib.moe_sample(logits.data_ptr(), _LOGITS[logits.dtype], M, V, logits.stride(0) if M > 1 else V, u.data_ptr(),
                        _raw(temperature), _raw(top_k), _raw(top_p), _raw(min_p), tokens.data_ptr(), _raw(probs),
                        _raw_stream(stream, dev))
    if rc:
        raise MoeError(rc, "moe_sample")

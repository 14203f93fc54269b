"""Python binding of the GB300 stack-wide paged-FP8 decode-attention library.

Argument marshalling only: every step of the decode path runs in the CUDA
kernels of ``libgk.so`` (sources in ``csrc/``, ABI in ``include/gk.h``).  There
is no CPU fallback: if the library cannot be built or loaded, or a tensor is not
on a CUDA device, the calls raise.

The functions carry the C names: ``gk_kv_append``, ``gk_decode_attn_stack``,
``gk_decode_step``, ``gk_decode_attn_stack_static``,
``gk_attn_workspace_bytes``, ``gk_attn_workspace_min_bytes``,
``gk_e4m3_quantize``, ``gk_kv_budget``, ``gk_kv_regions``, ``gk_kv_ingest``,
``gk_di_blocks``, ``gk_read_device_error``, ``gk_status_str``, ``gk_abi_version``; and, over a
4-bit cache (``include/gk_kv4.h``; a ``Kv4Cache`` or its tensors, ``new_kv4_cache``),
``gk_kv4_write``, ``gk_kv4_read``, ``gk_kv4_decode_attn_stack``, ``gk_kv4_decode_step``,
``gk_kv4_block_bytes``; and, for a prompt's pass (``include/gk_prompt.h``), ``gk_rope_table``,
``gk_rope``, ``gk_kv_write``, ``gk_kv_read``, ``gk_prompt_plan_bytes``, ``gk_prompt_plan``,
``gk_prompt_attn`` (plans: ``new_prompt_plan``).  Tensors are torch tensors; the stream defaults to torch's current stream
on the tensors' device.  The cache is a ``KvCache``: per-group
K and V buffers or stacked ``K_cache`` / ``V_cache``, exactly one of the two,
with packed-ness read from the K tensors' rank as the "GPT-OSS-120B giga-kernel
decode" page describes (section "KV-cache layout": ``k.dim() == v.dim() + 1``).
"""
from __future__ import annotations

import ctypes
import os
import re
import threading
from typing import Optional, Sequence

from . import build as _build

GK_OK, GK_ERR_INVALID_ARG, GK_ERR_UNSUPPORTED, GK_ERR_WORKSPACE, GK_ERR_CUDA, \
    GK_ERR_DEVICE_BOUNDS, GK_ERR_BUDGET = range(7)
GK_DEVERR_SLOT, GK_DEVERR_BLOCK, GK_DEVERR_POS, GK_DEVERR_TIMEOUT, GK_DEVERR_PLAN, \
    GK_DEVERR_INGEST = 0x1, 0x2, 0x4, 0x8, 0x10, 0x20
GK_K_PACKED, GK_K_PLAIN = 0, 1
GK_KV4_TILE_BYTES, GK_KV4_SKIP = 1152, -1
GK_KV_SKIP, GK_DEVERR_SEQ = -1, 0x40
GK_ROPE_PLAIN, GK_ROPE_LINEAR, GK_ROPE_YARN = 0, 1, 2
GK_ROPE_HALF, GK_ROPE_INTERLEAVED = 0, 1

HEADER = os.path.join(_build.INCLUDE, "gk.h")
KV4_HEADER = os.path.join(_build.INCLUDE, "gk_kv4.h")
PROMPT_HEADER = os.path.join(_build.INCLUDE, "gk_prompt.h")

_lock = threading.Lock()
_lib = None
_torch_module = None


class GkError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {gk_status_str(status)} ({status})")


class Shape(ctypes.Structure):
    """gk_shape: all int32."""
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_layers", "batch", "num_q_heads", "num_kv_heads", "head_dim",
        "block_size", "num_blocks", "window", "max_blocks_full", "max_blocks_swa")]

    @classmethod
    def make(cls, **kw) -> "Shape":
        return cls(**{k: int(v) for k, v in kw.items()})


class RopeParams(ctypes.Structure):
    """gk_rope_params; ``make`` takes the scaling by name ("none", "linear", "yarn") or number."""
    _fields_ = [("rot_dim", ctypes.c_int32), ("scaling", ctypes.c_int32)] + [
        (n, ctypes.c_double) for n in ("theta", "factor", "original_context", "beta_fast",
                                       "beta_slow")]
    SCALING = {"none": GK_ROPE_PLAIN, "linear": GK_ROPE_LINEAR, "yarn": GK_ROPE_YARN}

    @classmethod
    def make(cls, rot_dim, theta, scaling="none", factor=1.0, original_context=4096.0,
             beta_fast=32.0, beta_slow=1.0) -> "RopeParams":
        if scaling in cls.SCALING:
            scaling = cls.SCALING[scaling]
        elif isinstance(scaling, str):
            raise ValueError(f"scaling {scaling!r}: one of {sorted(cls.SCALING)}")
        return cls(int(rot_dim), int(scaling), float(theta), float(factor),
                   float(original_context), float(beta_fast), float(beta_slow))


class Prompt(ctypes.Structure):
    """gk_prompt: all int32."""
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_seqs", "num_q_heads", "num_kv_heads", "head_dim", "window", "q_tokens", "k_tokens")]


class KvRegion(ctypes.Structure):
    """gk_kv_region: one DI landing region (a group buffer's K or V half)."""
    _fields_ = [("base", ctypes.c_void_p), ("length", ctypes.c_uint64),
                ("block_len", ctypes.c_uint64)]


class KvCacheC(ctypes.Structure):
    """gk_kv_cache."""
    _fields_ = [("k_bufs", ctypes.c_void_p), ("v_bufs", ctypes.c_void_p),
                ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("k_layout", ctypes.c_int32)]


class KvCache:
    """The KV cache in one of its two forms ("Kernel contract": per-group
    buffers or stacked K_cache / V_cache, exactly one present).

    per-group: ``k_bufs[j]``, ``v_bufs[j]`` are group buffer j's K and V halves:
      V ``[num_blocks, kv, block, d]`` uint8, K the same (unpacked) or the packed
      view ``[num_blocks, kv, block // 2, d, 2]``;
    stacked: ``k_cache``, ``v_cache`` with a leading group axis (``[G, ...]``).
    ``k_layout`` is read from the ranks (``k.dim() == v.dim() + 1`` means packed);
    it must be given only when the buffers are raw device addresses (ints).
    Holds references to the tensors and the pointer arrays it hands the library.
    """

    def __init__(self, k_bufs=None, v_bufs=None, k_cache=None, v_cache=None,
                 k_layout: Optional[int] = None):
        per_group = k_bufs is not None or v_bufs is not None
        stacked = k_cache is not None or v_cache is not None
        if per_group == stacked:
            raise ValueError("pass exactly one KV form: (k_bufs, v_bufs) or (k_cache, v_cache)")
        if per_group and (k_bufs is None or v_bufs is None or len(k_bufs) != len(v_bufs)):
            raise ValueError("k_bufs and v_bufs must both be given, one per group buffer")
        if stacked and (k_cache is None or v_cache is None):
            raise ValueError("k_cache and v_cache must both be given")
        ks = list(k_bufs) if per_group else [k_cache]
        vs = list(v_bufs) if per_group else [v_cache]
        tensors = [(k, v) for k, v in zip(ks, vs) if not isinstance(k, int)
                   and not isinstance(v, int)]
        if tensors:
            inferred = {infer_k_layout(k, v) for k, v in tensors}
            if len(inferred) != 1:
                raise ValueError("all group buffers must have one K layout")
            inferred = inferred.pop()
            if k_layout is not None and k_layout != inferred:
                raise ValueError("k_layout disagrees with the K tensors' rank")
            k_layout = inferred
        elif k_layout is None:
            raise ValueError("k_layout is required for raw device addresses")
        if k_layout not in (GK_K_PACKED, GK_K_PLAIN):
            raise ValueError(f"k_layout {k_layout}")
        self.per_group = per_group
        self.k_layout = int(k_layout)
        self._keep = (ks, vs)
        self._held = None
        c = KvCacheC(k_layout=self.k_layout)
        if per_group:
            self._k_arr = _ptr_array(ks, "k_bufs")
            self._v_arr = _ptr_array(vs, "v_bufs")
            c.k_bufs = ctypes.cast(self._k_arr, ctypes.c_void_p)
            c.v_bufs = ctypes.cast(self._v_arr, ctypes.c_void_p)
        else:
            c.k_cache = _ptr(k_cache, None, "k_cache")
            c.v_cache = _ptr(v_cache, None, "v_cache")
        self.c = c

    def check(self, shape) -> None:
        """Buffer sizes against the shape (the C ABI cannot see them)."""
        sh = _as_shape(shape)
        groups = sh.num_layers // 2
        half = sh.num_blocks * sh.num_kv_heads * sh.block_size * sh.head_dim
        ks, vs = self._keep
        if self.per_group and len(ks) < groups:
            raise ValueError(f"{len(ks)} group buffers for {sh.num_layers} layers")
        want = half if self.per_group else groups * half
        for t in ks + vs:
            if not isinstance(t, int) and t.numel() * t.element_size() < want:
                raise ValueError(f"a cache buffer holds {t.numel() * t.element_size()} bytes, "
                                 f"the shape needs {want}")

    def held(self):
        """Of the buffers that are tensors: the smallest one's bytes, and their device (-1: several);
        (None, None) when there are none.  Looked up by the first call that asks."""
        if self._held is None:
            ts = [t for t in self._keep[0] + self._keep[1] if not isinstance(t, int)]
            devs = {t.get_device() for t in ts}
            self._held = (min((t.numel() * t.element_size() for t in ts), default=None),
                          None if not devs else devs.pop() if len(devs) == 1 else -1)
        return self._held

    def param(self):
        return ctypes.byref(self.c)


class Kv4CacheC(ctypes.Structure):
    """gk_kv4_cache."""
    _fields_ = [("bufs", ctypes.c_void_p), ("cache", ctypes.c_void_p)]


class Kv4Cache:
    """The 4-bit cache in one of its two forms, uint8 tensors on the device:

    per-group: a sequence of NL/2 group buffers [num_blocks, kv, block // 16, 1152];
    stacked:   one tensor with a leading group axis.
    Holds references to the tensors and the pointer array it hands the library;
    the calls take it, or the tensors themselves.
    """

    def __init__(self, bufs):
        self._stacked = hasattr(bufs, "data_ptr")
        self._keep = [bufs] if self._stacked else list(bufs)
        if not self._keep:
            raise ValueError("no group buffer")
        c = Kv4CacheC()
        if self._stacked:
            c.cache = _ptr(bufs, _torch().uint8, "kv")
        else:
            arr = (ctypes.c_void_p * len(self._keep))(
                *[_ptr(t, _torch().uint8, f"kv[{i}]") for i, t in enumerate(self._keep)])
            c.bufs = ctypes.cast(arr, ctypes.c_void_p)
            c.pointers = arr      # lives as long as the struct
        self.c = c

    def check(self, sh: Shape, dev: Optional[int] = None) -> None:
        """Buffer sizes against the shape, and their device (the C ABI cannot see them)."""
        groups, want = sh.num_layers // 2, _kv4_bytes(sh)
        if self._stacked:
            want *= groups
        elif len(self._keep) < groups:
            raise ValueError(f"{len(self._keep)} group buffers for {sh.num_layers} layers")
        for t in self._keep:
            if t.numel() < want:
                raise ValueError(f"a cache buffer holds {t.numel()} bytes, the shape needs {want}")
            if dev is not None and t.get_device() != dev:
                raise ValueError(f"a cache buffer is on cuda:{t.get_device()}, the current device "
                                 f"is cuda:{dev}")


def infer_k_layout(k, v) -> int:
    """Packed-ness from the ranks, as the page's bind step infers it
    (``k.dim() == v.dim() + 1``: the packed view's extra trailing axis of 2)."""
    kd, vd = k.dim(), v.dim()
    if kd == vd + 1 and k.shape[-1] == 2:
        return GK_K_PACKED
    if kd == vd:
        return GK_K_PLAIN
    raise ValueError(f"K shape {tuple(k.shape)} vs V shape {tuple(v.shape)}: "
                     "neither the packed view nor the plain layout")


def kv_from_group_buffers(bufs: Sequence, k_layout: int = GK_K_PACKED) -> KvCache:
    """Group buffers [2, num_blocks, kv, block, d] (K half, then V half) -> the
    per-group KvCache, K viewed packed ([.., block // 2, d, 2]) or plain."""
    ks = []
    for b in bufs:
        k = b[0]
        if k_layout == GK_K_PACKED:
            nb, kv, B, D = k.shape
            k = k.view(nb, kv, B // 2, D, 2)
        ks.append(k)
    return KvCache(k_bufs=ks, v_bufs=[b[1] for b in bufs])


def kv_stacked(k_cache, v_cache) -> KvCache:
    """Stacked K_cache / V_cache ([G, num_blocks, kv, block, d], K optionally
    as the packed view [G, num_blocks, kv, block // 2, d, 2])."""
    return KvCache(k_cache=k_cache, v_cache=v_cache)


def _kv(kv, shape) -> "ctypes._CArgObject":
    if not isinstance(kv, KvCache):
        raise TypeError("kv must be a KvCache (kv_from_group_buffers, kv_stacked)")
    kv.check(shape)
    return kv.param()


def _kv4_bytes(sh) -> int:
    """Bytes of one group buffer."""
    return sh.num_blocks * sh.num_kv_heads * (sh.block_size // 16) * GK_KV4_TILE_BYTES


def _kv4(kv, sh, dev):
    """The gk_kv4_cache of a Kv4Cache or of its tensors (which the caller holds)."""
    if hasattr(kv, "data_ptr"):
        return Kv4CacheC(None, _ptr4(kv, _torch().uint8, "kv", dev,
                                     sh.num_layers // 2 * _kv4_bytes(sh)))
    if not isinstance(kv, Kv4Cache):
        kv = Kv4Cache(kv)
    kv.check(sh, dev)
    return kv.c


def _current_device() -> int:
    try:
        return _torch()._C._cuda_getDevice()
    except RuntimeError:      # no driver: there are CPU tensors only, which are refused by name
        return 0


def _ptr4(t, dtype, name, dev, n, allow_none=False):
    """_ptr, of a tensor of at least n values that must lie on device `dev` (the current one: the
    library launches there)."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.numel() >= n:
            return t.data_ptr()
    except AttributeError:      # None or a raw address
        pass
    if t is None and allow_none:
        return None
    if hasattr(t, "get_device"):
        if t.is_cuda and t.get_device() != dev:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is "
                             f"cuda:{dev}")
        if t.numel() < n:
            raise ValueError(f"{name} holds {t.numel()} values, the call needs {n}")
    return _ptr(t, dtype, name)


def declared_functions(header: str = HEADER) -> list:
    """Names of the functions include/gk.h (or another header) declares."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(gk_[a-z0-9_]+)\s*\(", text)))


def lib(build_if_needed: bool = True) -> ctypes.CDLL:
    """Load libgk.so (building it with nvcc first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.build() if build_if_needed else _build.LIB_PATH
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: run paged_fp8_kv_gk_gb300.build.build()")
            L = ctypes.CDLL(path)
            vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
            sp = ctypes.POINTER(Shape)
            L.gk_status_str.restype = ctypes.c_char_p
            L.gk_status_str.argtypes = [ctypes.c_int]
            L.gk_abi_version.restype = i32
            L.gk_abi_version.argtypes = []
            L.gk_kv_append.restype = ctypes.c_int
            L.gk_kv_append.argtypes = [sp] + [vp] * 11
            L.gk_attn_workspace_bytes.restype = sz
            L.gk_attn_workspace_bytes.argtypes = [sp, vp]
            L.gk_attn_workspace_min_bytes.restype = sz
            L.gk_attn_workspace_min_bytes.argtypes = [sp]
            L.gk_decode_attn_stack.restype = ctypes.c_int
            L.gk_decode_attn_stack.argtypes = [sp] + [vp] * 15 + [sz, vp]
            L.gk_decode_step.restype = ctypes.c_int
            L.gk_decode_step.argtypes = [sp] + [vp] * 19 + [sz, vp]
            L.gk_decode_attn_stack_static.restype = ctypes.c_int
            L.gk_decode_attn_stack_static.argtypes = [sp] + [vp] * 15
            L.gk_e4m3_quantize.restype = ctypes.c_int
            L.gk_e4m3_quantize.argtypes = [vp, ctypes.c_float, vp, i64, vp]
            L.gk_kv_budget.restype = ctypes.c_int
            L.gk_kv_budget.argtypes = [ctypes.c_uint64, ctypes.c_uint64, ctypes.c_double,
                                       ctypes.c_double, ctypes.c_double, sp,
                                       ctypes.POINTER(ctypes.c_uint64),
                                       ctypes.POINTER(ctypes.c_int64)]
            L.gk_kv_regions.restype = ctypes.c_int
            L.gk_kv_regions.argtypes = [sp, vp, vp, ctypes.POINTER(KvRegion), i32,
                                        ctypes.POINTER(ctypes.c_int32)]
            L.gk_kv_ingest.restype = ctypes.c_int
            L.gk_kv_ingest.argtypes = [ctypes.POINTER(KvRegion), i32, vp, vp, i64, vp, vp]
            L.gk_di_blocks.restype = ctypes.c_int
            L.gk_di_blocks.argtypes = [i64, i32, i32] + [ctypes.POINTER(ctypes.c_int64)] * 3
            L.gk_kv4_block_bytes.restype = sz
            L.gk_kv4_block_bytes.argtypes = [sp]
            L.gk_kv4_write.restype = ctypes.c_int
            L.gk_kv4_write.argtypes = [sp, i32, i32, i64, vp, vp, i64, i64] + [vp] * 9
            L.gk_kv4_read.restype = ctypes.c_int
            L.gk_kv4_read.argtypes = [sp, i32, i32, i64] + [vp] * 9
            L.gk_kv4_decode_attn_stack.restype = ctypes.c_int
            L.gk_kv4_decode_attn_stack.argtypes = [sp] + [vp] * 15 + [sz, vp]
            L.gk_kv4_decode_step.restype = ctypes.c_int
            L.gk_kv4_decode_step.argtypes = [sp] + [vp] * 19 + [sz, vp]
            L.gk_rope_table.restype = ctypes.c_int
            L.gk_rope_table.argtypes = [ctypes.POINTER(RopeParams), i64] + [vp] * 4
            L.gk_rope.restype = ctypes.c_int
            L.gk_rope.argtypes = [i64, i32, i32, i32, i32, vp, i64, vp, vp, vp, i64, vp]
            L.gk_kv_write.restype = ctypes.c_int
            L.gk_kv_write.argtypes = [sp, i32, i32, i64, vp, vp, i64, i64] + [vp] * 9
            L.gk_kv_read.restype = ctypes.c_int
            L.gk_kv_read.argtypes = [sp, i32, i32, i64] + [vp] * 9
            pp = ctypes.POINTER(Prompt)
            L.gk_prompt_plan_bytes.restype = sz
            L.gk_prompt_plan_bytes.argtypes = [pp]
            L.gk_prompt_plan.restype = ctypes.c_int
            L.gk_prompt_plan.argtypes = [pp, vp, vp, vp, sz, vp]
            L.gk_prompt_attn.restype = ctypes.c_int
            L.gk_prompt_attn.argtypes = [pp, vp, sz, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp]
            L.gk_selftest_prompt_attn_timeout.restype = ctypes.c_int
            L.gk_selftest_prompt_attn_timeout.argtypes = [pp, vp, sz, vp, i64, vp, i64, vp, i64, vp, vp, vp,
                                                          i32, vp, ctypes.POINTER(ctypes.c_uint32)]
            L.gk_selftest_wait_timeout.restype = ctypes.c_int
            L.gk_selftest_wait_timeout.argtypes = [ctypes.c_uint64, vp,
                                                   ctypes.POINTER(ctypes.c_uint32)]
            L.gk_selftest_decode_attn_split.restype = ctypes.c_int
            L.gk_selftest_decode_attn_split.argtypes = [sp] + [vp] * 15 + [sz, i32, vp]
            L.gk_selftest_kv4_decode_attn_split.restype = ctypes.c_int
            L.gk_selftest_kv4_decode_attn_split.argtypes = [sp] + [vp] * 15 + [sz, i32, vp]
            L.gk_read_device_error.restype = ctypes.c_int
            L.gk_read_device_error.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), ctypes.c_int]
            _lib = L
    return _lib


# --------------------------------------------------------------- marshalling
def _ptr(t, dtype=None, name="tensor", allow_none=False):
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    return t.data_ptr()


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr_array(ts: Sequence, name: str):
    arr = (ctypes.c_void_p * len(ts))(*[_ptr(t, None, f"{name}[{i}]") for i, t in enumerate(ts)])
    return arr


def _stream(stream, like=None):
    if stream is None:
        torch = _torch()
        if like is not None and hasattr(like, "get_device"):
            return torch._C._cuda_getCurrentRawStream(like.get_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != GK_OK:
        raise GkError(status, where)


def _sinks(sinks, shape):
    """Optional attention-sink logits: fp32 [NL, Hq] on the device, or None."""
    import torch
    if sinks is None:
        return None
    if sinks.numel() != shape.num_layers * shape.num_q_heads:
        raise ValueError(f"sinks must hold num_layers * num_q_heads = "
                         f"{shape.num_layers * shape.num_q_heads} values")
    return _ptr(sinks, torch.float32, "sinks")


def _as_shape(shape) -> Shape:
    if isinstance(shape, Shape):
        return shape
    try:
        return Shape(**shape)
    except TypeError:      # values that are not plain ints
        return Shape.make(**shape)


# --------------------------------------------------------------- entry points
def gk_status_str(status: int) -> str:
    return lib().gk_status_str(int(status)).decode()


def gk_abi_version() -> int:
    return int(lib().gk_abi_version())


def gk_attn_workspace_bytes(shape) -> int:
    return int(lib().gk_attn_workspace_bytes(ctypes.byref(_as_shape(shape)), None))


def gk_attn_workspace_min_bytes(shape) -> int:
    return int(lib().gk_attn_workspace_min_bytes(ctypes.byref(_as_shape(shape))))


def gk_kv_append(shape, k_new, v_new, cos, sin, k_scale, v_scale, upd_full, upd_swa, active,
                 kv: KvCache, stream=None) -> None:
    import torch
    sh = _as_shape(shape)
    st = lib().gk_kv_append(
        ctypes.byref(sh), _ptr(k_new, torch.bfloat16, "k_new"), _ptr(v_new, torch.bfloat16, "v_new"),
        _ptr(cos, torch.float32, "cos"), _ptr(sin, torch.float32, "sin"),
        _ptr(k_scale, torch.float32, "k_scale"), _ptr(v_scale, torch.float32, "v_scale"),
        _ptr(upd_full, torch.int32, "upd_full"), _ptr(upd_swa, torch.int32, "upd_swa"),
        _ptr(active, torch.uint8, "active"), _kv(kv, sh), _stream(stream, k_new))
    _check(st, "gk_kv_append")


def gk_decode_attn_stack(shape, q, kv: KvCache, k_scale, v_scale, cos, sin, bt_full, bt_swa,
                         pos, pos_w, active, out, out_f32=None, workspace=None,
                         stream=None, sinks=None) -> None:
    import torch
    sh = _as_shape(shape)
    if workspace is None:
        raise ValueError("workspace is required (size: gk_attn_workspace_bytes(shape))")
    st = lib().gk_decode_attn_stack(
        ctypes.byref(sh), _ptr(q, torch.bfloat16, "q"), _kv(kv, sh),
        _ptr(k_scale, torch.float32, "k_scale"), _ptr(v_scale, torch.float32, "v_scale"),
        _ptr(cos, torch.float32, "cos"), _ptr(sin, torch.float32, "sin"),
        _ptr(bt_full, torch.int32, "bt_full"), _ptr(bt_swa, torch.int32, "bt_swa"),
        _ptr(pos, torch.int32, "pos"), _ptr(pos_w, torch.int32, "pos_w"),
        _ptr(active, torch.uint8, "active"), _sinks(sinks, sh), _ptr(out, torch.bfloat16, "out"),
        _ptr(out_f32, torch.float32, "out_f32", allow_none=True),
        _ptr(workspace, torch.uint8, "workspace"), int(workspace.numel()), _stream(stream, q))
    _check(st, "gk_decode_attn_stack")


def gk_decode_step(shape, q, k_new, v_new, cos, sin, k_scale, v_scale, upd_full, upd_swa,
                   bt_full, bt_swa, pos, pos_w, active, kv: KvCache, out, out_f32=None,
                   workspace=None, stream=None, sinks=None) -> None:
    """gk_kv_append + gk_decode_attn_stack in two launches (the append in the planner's)."""
    import torch
    sh = _as_shape(shape)
    if workspace is None:
        raise ValueError("workspace is required (size: gk_attn_workspace_bytes(shape))")
    st = lib().gk_decode_step(
        ctypes.byref(sh), _ptr(q, torch.bfloat16, "q"), _ptr(k_new, torch.bfloat16, "k_new"),
        _ptr(v_new, torch.bfloat16, "v_new"), _ptr(cos, torch.float32, "cos"),
        _ptr(sin, torch.float32, "sin"), _ptr(k_scale, torch.float32, "k_scale"),
        _ptr(v_scale, torch.float32, "v_scale"), _ptr(upd_full, torch.int32, "upd_full"),
        _ptr(upd_swa, torch.int32, "upd_swa"), _ptr(bt_full, torch.int32, "bt_full"),
        _ptr(bt_swa, torch.int32, "bt_swa"), _ptr(pos, torch.int32, "pos"),
        _ptr(pos_w, torch.int32, "pos_w"), _ptr(active, torch.uint8, "active"),
        _sinks(sinks, sh), _kv(kv, sh), _ptr(out, torch.bfloat16, "out"),
        _ptr(out_f32, torch.float32, "out_f32", allow_none=True),
        _ptr(workspace, torch.uint8, "workspace"), int(workspace.numel()), _stream(stream, q))
    _check(st, "gk_decode_step")


def gk_decode_attn_stack_static(shape, q, kv: KvCache, k_scale, v_scale, cos, sin, bt_full,
                                bt_swa, pos, pos_w, active, out, out_f32=None,
                                stream=None, sinks=None) -> None:
    """gk_decode_attn_stack without a caller workspace, for callers that cannot
    allocate device memory: the library's own fixed scratch array
    (GK_STATIC_SCRATCH_BYTES per GPU) serves as the workspace.  Calls on one
    device share that array, so they must not overlap on the GPU."""
    import torch
    sh = _as_shape(shape)
    st = lib().gk_decode_attn_stack_static(
        ctypes.byref(sh), _ptr(q, torch.bfloat16, "q"), _kv(kv, sh),
        _ptr(k_scale, torch.float32, "k_scale"), _ptr(v_scale, torch.float32, "v_scale"),
        _ptr(cos, torch.float32, "cos"), _ptr(sin, torch.float32, "sin"),
        _ptr(bt_full, torch.int32, "bt_full"), _ptr(bt_swa, torch.int32, "bt_swa"),
        _ptr(pos, torch.int32, "pos"), _ptr(pos_w, torch.int32, "pos_w"),
        _ptr(active, torch.uint8, "active"), _sinks(sinks, sh), _ptr(out, torch.bfloat16, "out"),
        _ptr(out_f32, torch.float32, "out_f32", allow_none=True), _stream(stream, q))
    _check(st, "gk_decode_attn_stack_static")


def gk_e4m3_quantize(x, scale: float, codes, stream=None) -> None:
    import torch
    st = lib().gk_e4m3_quantize(_ptr(x, torch.float32, "x"), float(scale),
                                _ptr(codes, torch.uint8, "codes"), int(x.numel()),
                                _stream(stream, x))
    _check(st, "gk_e4m3_quantize")


def gk_read_device_error(stream=None, clear: bool = True) -> int:
    """Synchronise the stream and return (and by default clear) the device
    error word: GK_DEVERR_* bits, 0 when nothing went out of range."""
    bits = ctypes.c_uint32(0)
    st = lib().gk_read_device_error(_stream(stream), ctypes.byref(bits), 1 if clear else 0)
    if st not in (GK_OK, GK_ERR_DEVICE_BOUNDS):
        raise GkError(st, "gk_read_device_error")
    return int(bits.value)


def gk_kv_budget(total_bytes: int, used_bytes: int, gpu_memory_utilization: float,
                 cap_fraction: float = 0.30, min_budget_gib: float = 1.0, shape=None):
    """KV pool size (host only): returns (status, available_bytes, num_blocks or None).
    GK_ERR_BUDGET is returned, not raised, so that callers can report the
    numbers the minimum-KV guard rejected."""
    avail = ctypes.c_uint64(0)
    nb = ctypes.c_int64(0)
    sh = ctypes.byref(_as_shape(shape)) if shape is not None else None
    st = lib().gk_kv_budget(int(total_bytes), int(used_bytes), float(gpu_memory_utilization),
                            float(cap_fraction), float(min_budget_gib), sh, ctypes.byref(avail),
                            ctypes.byref(nb) if shape is not None else None)
    if st not in (GK_OK, GK_ERR_BUDGET):
        raise GkError(st, "gk_kv_budget")
    return st, int(avail.value), (int(nb.value) if shape is not None else None)


def layer_binding(kv: KvCache, num_layers: int):
    """The per-layer binding of a KvCache (layer i -> group buffer i // 2), as
    device addresses: (layer_k, layer_v), each a list of num_layers ints."""
    ks, vs = kv._keep
    if kv.per_group:
        kb = [_ptr(t, None, "k") for t in ks]
        vb = [_ptr(t, None, "v") for t in vs]
    else:
        k, v = ks[0], vs[0]
        G = k.shape[0]
        half = k.numel() * k.element_size() // G
        kb = [_ptr(k, None, "k_cache") + j * half for j in range(G)]
        vb = [_ptr(v, None, "v_cache") + j * half for j in range(G)]
    return [kb[i // 2] for i in range(num_layers)], [vb[i // 2] for i in range(num_layers)]


def gk_kv_regions(shape, layer_k: Sequence[int], layer_v: Sequence[int]):
    """De-duplicated DI regions of a per-layer binding (host only): a ctypes
    array of KvRegion, K_0, V_0, K_1, V_1, ... for the page's layout."""
    sh = _as_shape(shape)
    n = len(layer_k)
    if n != sh.num_layers or len(layer_v) != n:
        raise ValueError("one K and one V address per layer")
    ka = (ctypes.c_void_p * n)(*layer_k)
    va = (ctypes.c_void_p * n)(*layer_v)
    cap = 2 * n
    out = (KvRegion * cap)()
    cnt = ctypes.c_int32(0)
    st = lib().gk_kv_regions(ctypes.byref(sh), ctypes.cast(ka, ctypes.c_void_p),
                             ctypes.cast(va, ctypes.c_void_p), out, cap, ctypes.byref(cnt))
    _check(st, "gk_kv_regions")
    return (KvRegion * cnt.value)(*out[:cnt.value])


def gk_kv_ingest(regions, dst_region, dst_block, src, stream=None) -> None:
    """Land len(dst_region) blocks from ``src`` (device tensor or pinned host
    tensor, n * block_len bytes) onto regions[dst_region[d]] block dst_block[d]."""
    import torch
    n = int(dst_region.numel())
    if int(dst_block.numel()) != n:
        raise ValueError("dst_region and dst_block must have one entry per descriptor")
    if n == 0:
        return
    if not src.is_contiguous():
        raise ValueError("src must be contiguous")
    if src.is_cuda is False and not src.is_pinned():
        raise ValueError("src must be a CUDA tensor or pinned host memory (no pageable copy)")
    bl = int(regions[0].block_len)
    if src.numel() * src.element_size() < n * bl:
        raise ValueError(f"src holds {src.numel() * src.element_size()} bytes, need {n * bl}")
    st = lib().gk_kv_ingest(regions, len(regions), _ptr(dst_region, torch.int32, "dst_region"),
                            _ptr(dst_block, torch.int32, "dst_block"), n, src.data_ptr(),
                            _stream(stream, dst_region))
    _check(st, "gk_kv_ingest")


def gk_di_blocks(num_tokens: int, block_size: int, window: int):
    """(full_count, swa_first, swa_count): the row blocks a decode engine needs
    for a prompt of num_tokens tokens, both engines operating at N - 1."""
    a, b, c = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    st = lib().gk_di_blocks(int(num_tokens), int(block_size), int(window), ctypes.byref(a),
                            ctypes.byref(b), ctypes.byref(c))
    _check(st, "gk_di_blocks")
    return a.value, b.value, c.value


# --------------------------------------------------------------- 4-bit cache
def gk_kv4_block_bytes(shape) -> int:
    return int(lib().gk_kv4_block_bytes(ctypes.byref(_as_shape(shape))))


def new_kv4_cache(shape, device="cuda", stacked: bool = True):
    """An uninitialised 4-bit cache of the shape: one tensor [NL/2, num_blocks, kv, block // 16,
    1152], or (stacked=False) a list of NL/2 group buffers.  No byte needs a value."""
    import torch
    sh = _as_shape(shape)
    if gk_kv4_block_bytes(sh) == 0:
        raise GkError(GK_ERR_UNSUPPORTED, "gk_kv4_block_bytes")
    size = (sh.num_blocks, sh.num_kv_heads, sh.block_size // 16, GK_KV4_TILE_BYTES)
    if stacked:
        return torch.empty((sh.num_layers // 2,) + size, dtype=torch.uint8, device=device)
    return [torch.empty(size, dtype=torch.uint8, device=device)
            for _ in range(sh.num_layers // 2)]


def _kv4_rows(sh, k, v, names, dev, contiguous):
    """Checks of a [layers, tokens, kv, 64] bf16 pair; returns (layers, tokens, strides)."""
    bf16 = _torch().bfloat16
    H, D = sh.num_kv_heads, sh.head_dim
    size = k.shape
    if k.is_contiguous() and v.is_contiguous() and k.dtype is bf16 and v.dtype is bf16 and \
            k.get_device() == dev == v.get_device() and size == v.shape and len(size) == 4 and \
            size[2] == H and size[3] == D:
        return size[0], size[1], (size[1] * H * D, H * D)
    for t, name in zip((k, v), names):
        if t.dtype != bf16:
            raise TypeError(f"{name}: expected {bf16}, got {t.dtype}")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is "
                             f"cuda:{dev}")
        if t.dim() != 4 or t.shape[2:] != (H, D):
            raise ValueError(f"{name} must be [layers, tokens, {H}, {D}]")
        if contiguous and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.numel() and (t.stride(3) != 1 or (H > 1 and t.stride(2) != D)):
            raise ValueError(f"{name}: the heads of a token must be contiguous")
    if size != v.shape:
        raise ValueError(f"{names[0]} and {names[1]} differ in shape")
    # the stride of an axis of one is never used
    sk = tuple(k.stride(a) if size[a] > 1 else 0 for a in (0, 1))
    sv = tuple(v.stride(a) if size[a] > 1 else 0 for a in (0, 1))
    if sk != sv:
        raise ValueError(f"{names[0]} and {names[1]} must have the same strides")
    return size[0], size[1], sk


def _kv4_step_args(sh, dev, q, k_scale, v_scale, cos, sin, bt_full, bt_swa, pos, pos_w, active,
                   sinks, out, out_f32, workspace, new=None):
    """The pointers that gk_kv4_decode_attn_stack and gk_kv4_decode_step share, in three runs: q;
    the scales and, for the step (new: k_new, v_new, upd_full, upd_swa), the new tokens around
    them; the control tensors and outputs."""
    torch = _torch()
    f32, i32, bf16 = torch.float32, torch.int32, torch.bfloat16
    NL, Bt = sh.num_layers, sh.batch
    rope, rows = Bt * sh.head_dim // 2, NL * Bt * sh.num_q_heads * sh.head_dim
    if workspace is None:
        raise ValueError("workspace is required (size: gk_attn_workspace_bytes(shape))")
    scales = [_ptr4(cos, f32, "cos", dev, rope), _ptr4(sin, f32, "sin", dev, rope)]
    ks = [_ptr4(k_scale, f32, "k_scale", dev, NL), _ptr4(v_scale, f32, "v_scale", dev, NL)]
    if new is None:
        head = [_ptr4(q, bf16, "q", dev, rows)]
        mid = ks + scales
    else:
        k_new, v_new, upd_full, upd_swa = new
        kv = NL * Bt * sh.num_kv_heads * sh.head_dim
        head = [_ptr4(q, bf16, "q", dev, rows), _ptr4(k_new, bf16, "k_new", dev, kv),
                _ptr4(v_new, bf16, "v_new", dev, kv)]
        mid = scales + ks + [_ptr4(upd_full, i32, "upd_full", dev, Bt),
                             _ptr4(upd_swa, i32, "upd_swa", dev, Bt)]
    if sinks is not None and sinks.numel() != NL * sh.num_q_heads:
        raise ValueError(f"sinks must hold num_layers * num_q_heads = "
                         f"{NL * sh.num_q_heads} values")
    mid += [_ptr4(bt_full, i32, "bt_full", dev, Bt * sh.max_blocks_full),
            _ptr4(bt_swa, i32, "bt_swa", dev, Bt * sh.max_blocks_swa),
            _ptr4(pos, i32, "pos", dev, Bt), _ptr4(pos_w, i32, "pos_w", dev, Bt),
            _ptr4(active, torch.uint8, "active", dev, Bt),
            _ptr4(sinks, f32, "sinks", dev, 1, True)]
    tail = [_ptr4(out, bf16, "out", dev, rows), _ptr4(out_f32, f32, "out_f32", dev, rows, True),
            _ptr4(workspace, torch.uint8, "workspace", dev, 1), workspace.numel()]
    return head, mid, tail


def gk_kv4_write(shape, k, v, cos, sin, k_scale, v_scale, slot_full, slot_swa, kv, active=None,
                 layer0: int = 0, stream=None) -> None:
    """Rotate, quantise and write the K and V of tokens into the 4-bit cache.

    k, v: bf16 [n_layers, n_tokens, kv, 64] of layers layer0 ..; the heads of a token are
    contiguous, layers and tokens may have any stride that is a multiple of 8.  cos, sin: fp32
    [n_tokens, 32], or both None for K that is rotated already.  slot_full, slot_swa: int32
    [n_tokens], GK_KV4_SKIP to leave a token out.  kv: a Kv4Cache or its tensors."""
    torch = _torch()
    f32, i32 = torch.float32, torch.int32
    sh, dev = _as_shape(shape), _current_device()
    n, T, (ls, ts) = _kv4_rows(sh, k, v, ("k", "v"), dev, False)
    kv = _kv4(kv, sh, dev)
    rope = T * sh.head_dim // 2
    st = lib().gk_kv4_write(
        ctypes.byref(sh), int(layer0), n, T, k.data_ptr(), v.data_ptr(), ls, ts,
        _ptr4(cos, f32, "cos", dev, rope, True), _ptr4(sin, f32, "sin", dev, rope, True),
        _ptr4(k_scale, f32, "k_scale", dev, sh.num_layers),
        _ptr4(v_scale, f32, "v_scale", dev, sh.num_layers),
        _ptr4(slot_full, i32, "slot_full", dev, T), _ptr4(slot_swa, i32, "slot_swa", dev, T),
        _ptr4(active, torch.uint8, "active", dev, T, True), ctypes.byref(kv), _stream(stream, k))
    _check(st, "gk_kv4_write")


def gk_kv4_read(shape, kv, k_scale, v_scale, slot_full, slot_swa, k_out, v_out, active=None,
                layer0: int = 0, stream=None) -> None:
    """The values at the given slots of the 4-bit cache, as bf16 [n_layers, n_tokens, kv, 64]
    (contiguous) of layers layer0 ..; the rows of skipped tokens are left as they were."""
    torch = _torch()
    f32, i32 = torch.float32, torch.int32
    sh, dev = _as_shape(shape), _current_device()
    n, T, _ = _kv4_rows(sh, k_out, v_out, ("k_out", "v_out"), dev, True)
    kv = _kv4(kv, sh, dev)
    st = lib().gk_kv4_read(
        ctypes.byref(sh), int(layer0), n, T, ctypes.byref(kv),
        _ptr4(k_scale, f32, "k_scale", dev, sh.num_layers),
        _ptr4(v_scale, f32, "v_scale", dev, sh.num_layers),
        _ptr4(slot_full, i32, "slot_full", dev, T), _ptr4(slot_swa, i32, "slot_swa", dev, T),
        _ptr4(active, torch.uint8, "active", dev, T, True), k_out.data_ptr(), v_out.data_ptr(),
        _stream(stream, k_out))
    _check(st, "gk_kv4_read")


def gk_kv4_decode_attn_stack(shape, q, kv, k_scale, v_scale, cos, sin, bt_full, bt_swa, pos,
                             pos_w, active, out, out_f32=None, workspace=None, stream=None,
                             sinks=None) -> None:
    """gk_decode_attn_stack over a 4-bit cache (a Kv4Cache or its tensors)."""
    sh, dev = _as_shape(shape), _current_device()
    head, mid, tail = _kv4_step_args(sh, dev, q, k_scale, v_scale, cos, sin, bt_full, bt_swa, pos,
                                     pos_w, active, sinks, out, out_f32, workspace)
    kv = _kv4(kv, sh, dev)
    st = lib().gk_kv4_decode_attn_stack(ctypes.byref(sh), *head, ctypes.byref(kv), *mid, *tail,
                                        _stream(stream, q))
    _check(st, "gk_kv4_decode_attn_stack")


def gk_kv4_decode_step(shape, q, k_new, v_new, cos, sin, k_scale, v_scale, upd_full, upd_swa,
                       bt_full, bt_swa, pos, pos_w, active, kv, out, out_f32=None,
                       workspace=None, stream=None, sinks=None) -> None:
    """gk_kv4_write of every row's new token + gk_kv4_decode_attn_stack in two launches."""
    sh, dev = _as_shape(shape), _current_device()
    head, mid, tail = _kv4_step_args(sh, dev, q, k_scale, v_scale, cos, sin, bt_full, bt_swa, pos,
                                     pos_w, active, sinks, out, out_f32, workspace,
                                     (k_new, v_new, upd_full, upd_swa))
    kv = _kv4(kv, sh, dev)
    st = lib().gk_kv4_decode_step(ctypes.byref(sh), *head, *mid, ctypes.byref(kv), *tail,
                                  _stream(stream, q))
    _check(st, "gk_kv4_decode_step")


# --------------------------------------------------------------- a prompt's pass
def gk_rope_table(params, pos, cos, sin, stream=None) -> None:
    """cos and sin, fp32 [n, rot_dim / 2], of the positions `pos` (int32 [n]).  params: a RopeParams
    or its fields (rot_dim, theta, scaling "none", "linear" or "yarn", factor, ...)."""
    torch = _torch()
    dev = _current_device()
    if not isinstance(params, RopeParams):
        params = RopeParams.make(**params)
    n = pos.numel()
    want = n * params.rot_dim // 2
    st = lib().gk_rope_table(
        ctypes.byref(params), n, _ptr4(pos, torch.int32, "pos", dev, n),
        _ptr4(cos, torch.float32, "cos", dev, want), _ptr4(sin, torch.float32, "sin", dev, want),
        _stream(stream, pos))
    _check(st, "gk_rope_table")


def _heads(t, name, dev, heads=None, dim=None):
    """Checks of a bf16 [tokens, heads, channels] tensor with contiguous heads, as slices of a fused
    projection are; returns (tokens, heads, channels, token stride)."""
    size, stride = t.shape, t.stride()
    if len(size) == 3 and t.dtype is _torch().bfloat16 and t.get_device() == dev:
        T, H, D = size
        if stride[2] == 1 and stride[1] == D and T > 1 and (heads is None or (H == heads and D == dim)):
            return T, H, D, stride[0]
    if t.dtype is not _torch().bfloat16:
        raise TypeError(f"{name}: expected {_torch().bfloat16}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{dev}")
    if len(size) != 3 or (heads is not None and size[1:] != (heads, dim)):
        raise ValueError(f"{name} must be [tokens, "
                         f"{'heads, channels' if heads is None else f'{heads}, {dim}'}]")
    T, H, D = size
    if t.numel() and ((D > 1 and stride[2] != 1) or (H > 1 and stride[1] != D)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return T, H, D, stride[0] if T > 1 else H * D


def gk_rope(x, cos, sin, out, layout="half", stream=None) -> None:
    """Rotate the heads of x by cos and sin (fp32 [n, rot_dim / 2]; channels from rot_dim on are
    copied) into out, which may be x.  x, out: bf16 [n, heads, head_dim], the heads of a token
    contiguous, tokens of any stride that is a multiple of 8.  layout: "half" (pairs e, e +
    rot_dim / 2) or "interleaved" (pairs 2e, 2e + 1)."""
    torch = _torch()
    dev = _current_device()
    n, H, D, xs = _heads(x, "x", dev)
    m, _, _, os_ = _heads(out, "out", dev, H, D)
    if m != n:
        raise ValueError(f"out has {m} tokens, x has {n}")
    if layout not in ("half", "interleaved"):
        raise ValueError(f"layout {layout!r}: 'half' or 'interleaved'")
    if cos.dim() != 2 or cos.shape[0] != n or sin.shape != cos.shape:
        raise ValueError(f"cos and sin must be [{n}, rot_dim / 2]")
    rot = 2 * cos.shape[1]
    st = lib().gk_rope(
        n, H, D, rot, GK_ROPE_HALF if layout == "half" else GK_ROPE_INTERLEAVED, x.data_ptr(), xs,
        _ptr4(cos, torch.float32, "cos", dev, 0), _ptr4(sin, torch.float32, "sin", dev, 0),
        out.data_ptr(), os_, _stream(stream, x))
    _check(st, "gk_rope")


def _kv_on(kv, sh, dev):
    """The gk_kv_cache of a KvCache whose tensors must lie on device `dev` (the current one: the
    library launches there) and hold the shape."""
    if not isinstance(kv, KvCache):
        raise TypeError("kv must be a KvCache (kv_from_group_buffers, kv_stacked)")
    groups = sh.num_layers // 2
    half = sh.num_blocks * sh.num_kv_heads * sh.block_size * sh.head_dim
    held, on = kv.held()
    if on is not None and on != dev:
        raise ValueError(f"the cache buffers are not all on the current device, cuda:{dev}")
    if (kv.per_group and len(kv._keep[0]) < groups) or (
            held is not None and held < (half if kv.per_group else groups * half)):
        kv.check(sh)       # names what is wrong
    return kv.param()


def gk_kv_write(shape, k, v, cos, sin, k_scale, v_scale, slot_full, slot_swa, kv: KvCache,
                active=None, layer0: int = 0, stream=None) -> None:
    """Rotate, quantise and write the K and V of tokens into the FP8 cache.

    k, v: bf16 [n_layers, n_tokens, kv, 64] of layers layer0 ..; the heads of a token are
    contiguous, layers and tokens may have any stride that is a multiple of 8.  cos, sin: fp32
    [n_tokens, 32], or both None for K that is rotated already.  slot_full, slot_swa: int32
    [n_tokens], GK_KV_SKIP to leave a token out."""
    torch = _torch()
    f32, i32 = torch.float32, torch.int32
    sh, dev = _as_shape(shape), _current_device()
    n, T, (ls, ts) = _kv4_rows(sh, k, v, ("k", "v"), dev, False)
    rope = T * sh.head_dim // 2
    st = lib().gk_kv_write(
        ctypes.byref(sh), int(layer0), n, T, k.data_ptr(), v.data_ptr(), ls, ts,
        _ptr4(cos, f32, "cos", dev, rope, True), _ptr4(sin, f32, "sin", dev, rope, True),
        _ptr4(k_scale, f32, "k_scale", dev, sh.num_layers),
        _ptr4(v_scale, f32, "v_scale", dev, sh.num_layers),
        _ptr4(slot_full, i32, "slot_full", dev, T), _ptr4(slot_swa, i32, "slot_swa", dev, T),
        _ptr4(active, torch.uint8, "active", dev, T, True), _kv_on(kv, sh, dev),
        _stream(stream, k))
    _check(st, "gk_kv_write")


def gk_kv_read(shape, kv: KvCache, k_scale, v_scale, slot_full, slot_swa, k_out, v_out,
               active=None, layer0: int = 0, stream=None) -> None:
    """The values at the given slots of the FP8 cache, as bf16 [n_layers, n_tokens, kv, 64]
    (contiguous) of layers layer0 ..; the rows of skipped tokens are left as they were."""
    torch = _torch()
    f32, i32 = torch.float32, torch.int32
    sh, dev = _as_shape(shape), _current_device()
    n, T, _ = _kv4_rows(sh, k_out, v_out, ("k_out", "v_out"), dev, True)
    st = lib().gk_kv_read(
        ctypes.byref(sh), int(layer0), n, T, _kv_on(kv, sh, dev),
        _ptr4(k_scale, f32, "k_scale", dev, sh.num_layers),
        _ptr4(v_scale, f32, "v_scale", dev, sh.num_layers),
        _ptr4(slot_full, i32, "slot_full", dev, T), _ptr4(slot_swa, i32, "slot_swa", dev, T),
        _ptr4(active, torch.uint8, "active", dev, T, True), k_out.data_ptr(), v_out.data_ptr(),
        _stream(stream, k_out))
    _check(st, "gk_kv_read")


def _as_prompt(prompt) -> Prompt:
    if isinstance(prompt, Prompt):
        return prompt
    try:
        return Prompt(**prompt)
    except TypeError:      # values that are not plain ints
        return Prompt(**{k: int(v) for k, v in prompt.items()})


def gk_prompt_plan_bytes(prompt) -> int:
    return int(lib().gk_prompt_plan_bytes(ctypes.byref(_as_prompt(prompt))))


def new_prompt_plan(prompt, device="cuda"):
    """Room for the plan of a prompt's attention (gk_prompt_plan fills it)."""
    import torch
    n = gk_prompt_plan_bytes(prompt)
    if n == 0:
        raise GkError(GK_ERR_UNSUPPORTED, "gk_prompt_plan_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def gk_prompt_plan(prompt, q_start, k_start, plan, stream=None) -> None:
    """Work out the tiles of a prompt's attention from the sequences' starts (int32 [num_seqs + 1] on
    the device), for every layer with these sequences and this window.  prompt: a Prompt or its
    fields."""
    torch = _torch()
    pr, dev = _as_prompt(prompt), _current_device()
    st = lib().gk_prompt_plan(
        ctypes.byref(pr), _ptr4(q_start, torch.int32, "q_start", dev, pr.num_seqs + 1),
        _ptr4(k_start, torch.int32, "k_start", dev, pr.num_seqs + 1),
        _ptr4(plan, torch.uint8, "plan", dev, 1), plan.numel(), _stream(stream, q_start))
    _check(st, "gk_prompt_plan")


def _prompt_args(prompt, plan, q, k, v, out, out_f32, sinks):
    """gk_prompt_attn's arguments up to the stream."""
    torch = _torch()
    pr, dev = _as_prompt(prompt), _current_device()
    Hq, H, D = pr.num_q_heads, pr.num_kv_heads, pr.head_dim
    strides = []
    for t, name, rows, heads in ((q, "q", pr.q_tokens, Hq), (k, "k", pr.k_tokens, H),
                                 (v, "v", pr.k_tokens, H)):
        T, _, _, s = _heads(t, name, dev, heads, D)
        if T < rows:
            raise ValueError(f"{name} has {T} tokens, the prompt {rows}")
        strides.append(s)
    if sinks is not None and sinks.numel() != Hq:
        raise ValueError(f"sinks must hold num_q_heads = {Hq} values")
    n = pr.q_tokens * Hq * D
    return (ctypes.byref(pr), _ptr4(plan, torch.uint8, "plan", dev, 1), plan.numel(), q.data_ptr(),
            strides[0], k.data_ptr(), strides[1], v.data_ptr(), strides[2],
            _ptr4(sinks, torch.float32, "sinks", dev, 1, True),
            _ptr4(out, torch.bfloat16, "out", dev, n),
            _ptr4(out_f32, torch.float32, "out_f32", dev, n, True))


def gk_prompt_attn(prompt, plan, q, k, v, out, out_f32=None, sinks=None, stream=None) -> None:
    """Causal attention of packed sequences, one layer, along a plan of gk_prompt_plan.

    q: bf16 [q_tokens, q heads, 64]; k, v: bf16 [k_tokens, kv heads, 64]; the heads of a token are
    contiguous, tokens may have any stride that is a multiple of 8.  out (bf16) and out_f32 are
    contiguous; their rows outside every sequence are left as they were; they may not overlap the other
    tensors.  sinks: fp32 [q heads]."""
    st = lib().gk_prompt_attn(*_prompt_args(prompt, plan, q, k, v, out, out_f32, sinks),
                              _stream(stream, q))
    _check(st, "gk_prompt_attn")


def gk_selftest_prompt_attn_timeout(prompt, plan, q, k, v, out, out_f32=None, sinks=None,
                                    wait_tries: int = 1 << 18, stream=None) -> int:
    """Test hook (include/gk_testing.h): gk_prompt_attn whose waits run out; returns the device error
    word (GK_DEVERR_TIMEOUT expected)."""
    bits = ctypes.c_uint32(0)
    st = lib().gk_selftest_prompt_attn_timeout(
        *_prompt_args(prompt, plan, q, k, v, out, out_f32, sinks), int(wait_tries),
        _stream(stream, q), ctypes.byref(bits))
    if st not in (GK_OK, GK_ERR_DEVICE_BOUNDS):
        raise GkError(st, "gk_selftest_prompt_attn_timeout")
    return int(bits.value)


def gk_selftest_wait_timeout(limit_ns: int, stream=None) -> int:
    """Test hook (include/gk_testing.h): run the bounded barrier wait into its
    limit on the GPU; returns the device error word (GK_DEVERR_TIMEOUT expected)."""
    bits = ctypes.c_uint32(0)
    st = lib().gk_selftest_wait_timeout(int(limit_ns), _stream(stream), ctypes.byref(bits))
    if st not in (GK_OK, GK_ERR_DEVICE_BOUNDS):
        raise GkError(st, "gk_selftest_wait_timeout")
    return int(bits.value)


def gk_selftest_decode_attn_split(shape, q, kv: KvCache, k_scale, v_scale, cos, sin, bt_full,
                                  bt_swa, pos, pos_w, active, out, out_f32, workspace,
                                  split_tokens: int, stream=None, sinks=None) -> None:
    """Test hook (include/gk_testing.h): gk_decode_attn_stack with the split-KV
    chunk length fixed to `split_tokens` (a power of two >= 512)."""
    import torch
    sh = _as_shape(shape)
    st = lib().gk_selftest_decode_attn_split(
        ctypes.byref(sh), _ptr(q, torch.bfloat16, "q"), _kv(kv, sh),
        _ptr(k_scale, torch.float32, "k_scale"), _ptr(v_scale, torch.float32, "v_scale"),
        _ptr(cos, torch.float32, "cos"), _ptr(sin, torch.float32, "sin"),
        _ptr(bt_full, torch.int32, "bt_full"), _ptr(bt_swa, torch.int32, "bt_swa"),
        _ptr(pos, torch.int32, "pos"), _ptr(pos_w, torch.int32, "pos_w"),
        _ptr(active, torch.uint8, "active"), _sinks(sinks, sh), _ptr(out, torch.bfloat16, "out"),
        _ptr(out_f32, torch.float32, "out_f32", allow_none=True),
        _ptr(workspace, torch.uint8, "workspace"), int(workspace.numel()), int(split_tokens),
        _stream(stream, q))
    _check(st, "gk_selftest_decode_attn_split")


def gk_selftest_kv4_decode_attn_split(shape, q, kv, k_scale, v_scale, cos, sin, bt_full, bt_swa,
                                      pos, pos_w, active, out, out_f32, workspace,
                                      split_tokens: int, stream=None, sinks=None) -> None:
    """Test hook (include/gk_testing.h): gk_kv4_decode_attn_stack with the split-KV chunk length
    fixed to `split_tokens` (a power of two >= 512)."""
    sh, dev = _as_shape(shape), _current_device()
    head, mid, tail = _kv4_step_args(sh, dev, q, k_scale, v_scale, cos, sin, bt_full, bt_swa, pos,
                                     pos_w, active, sinks, out, out_f32, workspace)
    kv = _kv4(kv, sh, dev)
    st = lib().gk_selftest_kv4_decode_attn_split(ctypes.byref(sh), *head, ctypes.byref(kv), *mid,
                                                 *tail, int(split_tokens), _stream(stream, q))
    _check(st, "gk_selftest_kv4_decode_attn_split")


def new_workspace(shape, device="cuda"):
    import torch
    n = gk_attn_workspace_bytes(shape)
    if n == 0:
        raise GkError(GK_ERR_UNSUPPORTED, "gk_attn_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)

"""Python binding of libfdllm.so, the C-ABI library of the Fast-dLLM step.

Argument marshalling only: every computation runs in the library's CUDA
kernels. torch provides device memory (outputs and scratch are allocated as
torch tensors) and the current CUDA stream. If the shared object is missing,
every call raises: there is no fallback of any kind.

Layouts follow include/fdllm.h:
  q, out   [b, B, Hq, d]     k_cache, v_cache [b, Hkv, L, d]
  h        [M, D]            w [V, D]
  conf/tok [b, B]            x [b, L] int32, masked [b, L] uint8
"""
from __future__ import annotations

import ctypes
import os

import torch

# FDLLM_LIB may name another build of the library (the instrumented
# libfdllm_timeline.so of `python -m block_kv_cache_b200.build --timeline`).
LIB_PATH = os.environ.get("FDLLM_LIB") or os.path.join(os.path.dirname(os.path.abspath(__file__)),
                                                       "libfdllm.so")

FDL_OK, FDL_EINVAL, FDL_EUNSUPPORTED, FDL_ECUDA, FDL_ETIMEOUT, FDL_EWORKSPACE, FDL_EDEVICE = (
    0, -1, -2, -3, -4, -5, -6)
FDL_F32, FDL_BF16 = 0, 1

EXPORTS = ("fdl_abi_version", "fdl_create", "fdl_destroy", "fdl_last_error",
           "fdl_get_device_status", "fdl_set_wait_timeout", "fdl_attention_workspace_bytes",
           "fdl_dualcache_attention", "fdl_kv_store", "fdl_lmhead_workspace_bytes",
           "fdl_lmhead_confidence", "fdl_threshold_unmask",
           "fdl_lmhead_confidence_noalloc", "fdl_rope_table", "fdl_rmsnorm", "fdl_embed",
           "fdl_qkv_rope_store", "fdl_linear_residual", "fdl_linear_swiglu",
           "fdl_full_attention", "fdl_ffn", "fdl_qkv_attention", "fdl_model_create",
           "fdl_model_destroy", "fdl_generate_workspace_bytes", "fdl_generate",
           "fdl_kv4_store", "fdl_kv4_load", "fdl_kv4_attention_workspace_bytes",
           "fdl_kv4_attention_plan", "fdl_kv4_attention", "fdl_generate_workspace_bytes_kv")


class AttnDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("n_q_heads", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("seq_len", ctypes.c_int), ("block_start", ctypes.c_int),
                ("block_len", ctypes.c_int), ("dtype", ctypes.c_int),
                ("scale", ctypes.c_float)]


ABI_VERSION = 8
KV4_MAX_SEQ = 1 << 30


class Kv4Buffers(ctypes.Structure):
    """fdl_kv4_cache."""
    _fields_ = [("k", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


class Kv4RowsDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("seq_len", ctypes.c_int), ("dtype", ctypes.c_int),
                ("seq_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class Kv4AttnDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("n_q_heads", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("seq_len", ctypes.c_int), ("block_start", ctypes.c_int),
                ("block_len", ctypes.c_int), ("dtype", ctypes.c_int),
                ("scale", ctypes.c_float), ("window_left", ctypes.c_int),
                ("window_right", ctypes.c_int), ("sinks", ctypes.c_int)]


class Kv4Plan(ctypes.Structure):
    """fdl_kv4_plan: which kernel takes an attention over a 4-bit cache, and its splits."""
    _fields_ = [("many_rows", ctypes.c_int), ("row_tiles", ctypes.c_int),
                ("splits", ctypes.c_int), ("cluster", ctypes.c_int)]


class LMHeadDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("hidden", ctypes.c_int),
                ("vocab", ctypes.c_int), ("dtype", ctypes.c_int)]


class UnmaskDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("seq_len", ctypes.c_int),
                ("block_start", ctypes.c_int), ("block_len", ctypes.c_int),
                ("tau", ctypes.c_float)]


class QKVDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("hidden", ctypes.c_int), ("n_q_heads", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("batch", ctypes.c_int), ("seq_len", ctypes.c_int),
                ("rows_per_seq", ctypes.c_int), ("pos0", ctypes.c_int),
                ("max_pos", ctypes.c_int)]


class ModelDesc(ctypes.Structure):
    _fields_ = [("vocab", ctypes.c_int), ("hidden", ctypes.c_int), ("n_layers", ctypes.c_int),
                ("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("ffn", ctypes.c_int), ("mask_id", ctypes.c_int),
                ("rope_theta", ctypes.c_float), ("rms_eps", ctypes.c_float)]


class LayerWeights(ctypes.Structure):
    _fields_ = [("attn_norm", ctypes.c_void_p), ("w_qkv", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("wo", ctypes.c_void_p),
                ("ffn_norm", ctypes.c_void_p), ("w_gu", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p)]


class ModelWeights(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("final_norm", ctypes.c_void_p),
                ("lm_head", ctypes.c_void_p), ("layers", ctypes.POINTER(LayerWeights))]


FDL_CACHE_DUAL, FDL_CACHE_PREFIX, FDL_CACHE_NONE = 0, 1, 2
CACHE_MODES = {"dual": FDL_CACHE_DUAL, "prefix": FDL_CACHE_PREFIX, "none": FDL_CACHE_NONE}


class GenerateOpts(ctypes.Structure):
    _fields_ = [("cache", ctypes.c_int), ("device_loop", ctypes.c_int),
                ("bias_tok", ctypes.c_void_p), ("bias_val", ctypes.c_void_p),
                ("batching", ctypes.c_int), ("kv", ctypes.c_int)]


KV_FORMATS = {"bf16": 0, "4bit": 1}
BATCHING = {"lockstep": 0, "compact": 1, "per_sequence": 2}


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # none in a CPU build


class FdlError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"fdllm error {code}: {msg}")
        self.code = code


_lib = None


def load() -> ctypes.CDLL:
    """Load libfdllm.so and declare its signatures (raises if not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m block_kv_cache_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.fdl_abi_version.restype = i
    if L.fdl_abi_version() != ABI_VERSION:
        raise RuntimeError(f"{LIB_PATH} has ABI {L.fdl_abi_version()}, this binding expects "
                           f"{ABI_VERSION}: rebuild with `python -m block_kv_cache_b200.build`")
    L.fdl_create.argtypes = [ctypes.POINTER(vp), i]
    L.fdl_destroy.argtypes = [vp]
    L.fdl_last_error.restype = ctypes.c_char_p
    L.fdl_get_device_status.argtypes = [vp, vp]
    L.fdl_set_wait_timeout.argtypes = [vp, ctypes.c_uint64]
    L.fdl_attention_workspace_bytes.argtypes = [vp, ctypes.POINTER(AttnDesc)]
    L.fdl_attention_workspace_bytes.restype = sz
    L.fdl_dualcache_attention.argtypes = [vp, ctypes.POINTER(AttnDesc), vp, vp, vp, vp, vp,
                                          vp, sz, vp]
    L.fdl_kv_store.argtypes = [vp, ctypes.POINTER(AttnDesc), vp, vp, i, i, vp, vp, vp]
    L.fdl_lmhead_workspace_bytes.argtypes = [vp, ctypes.POINTER(LMHeadDesc)]
    L.fdl_lmhead_workspace_bytes.restype = sz
    L.fdl_lmhead_confidence.argtypes = [vp, ctypes.POINTER(LMHeadDesc), vp, vp, vp, vp, vp,
                                        vp, vp, sz, vp]
    L.fdl_lmhead_confidence_noalloc.argtypes = [vp, ctypes.POINTER(LMHeadDesc), vp, vp, vp, vp,
                                                vp, vp, vp]
    L.fdl_threshold_unmask.argtypes = [vp, ctypes.POINTER(UnmaskDesc), vp, vp, vp, vp, vp,
                                       vp, vp]
    L.fdl_rope_table.argtypes = [ctypes.c_double, i, i, vp]
    L.fdl_rmsnorm.argtypes = [vp, i, i, vp, vp, vp, ctypes.c_float, vp, vp]
    L.fdl_embed.argtypes = [vp, i, i, vp, vp, vp, vp, vp]
    L.fdl_qkv_rope_store.argtypes = [vp, ctypes.POINTER(QKVDesc), vp, vp, vp, vp, vp, vp, vp, vp]
    L.fdl_linear_residual.argtypes = [vp, i, i, i, vp, vp, vp, vp]
    L.fdl_linear_swiglu.argtypes = [vp, i, i, i, vp, vp, vp, vp]
    L.fdl_full_attention.argtypes = [vp, ctypes.POINTER(AttnDesc), vp, vp, vp, vp, vp]
    fl = ctypes.c_float
    L.fdl_ffn.argtypes = [vp, i, i, i, vp, fl, vp, vp, vp, vp, vp, vp]
    L.fdl_qkv_attention.argtypes = [vp, ctypes.POINTER(QKVDesc), vp, vp, fl, vp, vp, vp, vp, vp,
                                    vp, vp, vp, vp]
    L.fdl_model_create.argtypes = [ctypes.POINTER(ModelDesc), ctypes.POINTER(ModelWeights),
                                   ctypes.POINTER(vp)]
    L.fdl_model_destroy.argtypes = [vp]
    L.fdl_generate_workspace_bytes.argtypes = [vp, vp, i, i, i]
    L.fdl_generate_workspace_bytes.restype = sz
    L.fdl_generate_workspace_bytes_kv.argtypes = [vp, vp, i, i, i, i]
    L.fdl_generate_workspace_bytes_kv.restype = sz
    L.fdl_generate.argtypes = [vp, vp, vp, i, i, i, i, fl, ctypes.POINTER(GenerateOpts), vp,
                               ctypes.POINTER(i), vp, sz, vp]
    L.fdl_kv4_store.argtypes = [vp, ctypes.POINTER(Kv4RowsDesc), vp, vp, i, i,
                                ctypes.POINTER(Kv4Buffers), vp]
    L.fdl_kv4_load.argtypes = [vp, ctypes.POINTER(Kv4RowsDesc), ctypes.POINTER(Kv4Buffers), i, i,
                               vp, vp, vp]
    L.fdl_kv4_attention_workspace_bytes.argtypes = [vp, ctypes.POINTER(Kv4AttnDesc)]
    L.fdl_kv4_attention_workspace_bytes.restype = sz
    L.fdl_kv4_attention_plan.argtypes = [vp, ctypes.POINTER(Kv4AttnDesc), ctypes.POINTER(Kv4Plan)]
    L.fdl_kv4_attention.argtypes = [vp, ctypes.POINTER(Kv4AttnDesc), vp,
                                    ctypes.POINTER(Kv4Buffers), vp, vp, vp, vp, sz, vp]
    for name in EXPORTS:
        getattr(L, name).restype = getattr(L, name).restype or i
    _lib = L
    return L


def _check(rc: int):
    if rc != FDL_OK:
        raise FdlError(rc, load().fdl_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return FDL_F32
    if t.dtype == torch.bfloat16:
        return FDL_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _need(t: torch.Tensor, name: str, dtype=None, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def rope_table(theta: float, max_pos: int, head_dim: int):
    """(cos, sin) table of rotate-half RoPE as a host float32 array [max_pos, head_dim/2, 2]
    (computed by the library in double precision)."""
    import numpy as np
    out = np.empty((max_pos, head_dim // 2, 2), np.float32)
    _check(load().fdl_rope_table(float(theta), int(max_pos), int(head_dim),
                                 ctypes.c_void_p(out.ctypes.data)))
    return out


_I32 = 1 << 31


def _i32(x, name):
    """An int argument of a call; ctypes would drop the bits above 32."""
    x = int(x)
    if not -_I32 <= x < _I32:
        raise ValueError(f"{name} {x} does not fit in 32 bits")
    return x


class Kv4Cache:
    """One layer's K/V cache in microscaled 4-bit floating point (fdl_kv4_cache): codes k, v
    [b, Hkv, L, d/2] and scales k_scale, v_scale [b, Hkv, L, d/16], uint8 CUDA tensors that the
    caller may own (Kv4Cache(k, k_scale, v, v_scale)) or have allocated here (Kv4Cache.empty,
    zeroed: every position reads as 0 until it is stored). It stays with these tensors and
    their memory: another Kv4Cache is made for others."""
    k = property(lambda self: self._tensors[0])
    k_scale = property(lambda self: self._tensors[1])
    v = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])

    def __init__(self, k, k_scale, v, v_scale):
        try:
            b, h, L, half = shape = k.shape
            scales, dev, u8 = (b, h, L, half // 8), k.get_device(), torch.uint8
            right = ((half == 64 or half == 32) and dev >= 0 and L <= KV4_MAX_SEQ
                     and b <= KV4_MAX_SEQ and h <= KV4_MAX_SEQ
                     and v.shape == shape and k_scale.shape == scales and v_scale.shape == scales
                     and k.dtype is u8 and k_scale.dtype is u8 and v.dtype is u8
                     and v_scale.dtype is u8 and k_scale.get_device() == dev
                     and v.get_device() == dev and v_scale.get_device() == dev
                     and k.is_contiguous() and k_scale.is_contiguous() and v.is_contiguous()
                     and v_scale.is_contiguous())
        except (AttributeError, ValueError):
            right = False
        if not right:
            self._refuse(k, k_scale, v, v_scale)
        self._tensors = k, k_scale, v, v_scale
        self.batch, self.n_kv_heads, self.seq_len, self.head_dim = b, h, L, 2 * half
        self.device_index = dev
        self.buffers = Kv4Buffers(k.data_ptr(), k_scale.data_ptr(), v.data_ptr(),
                                  v_scale.data_ptr())

    @staticmethod
    def _refuse(k, k_scale, v, v_scale):
        for t, n in ((k, "k"), (k_scale, "k_scale"), (v, "v"), (v_scale, "v_scale")):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype is not torch.uint8 \
                    or not t.is_contiguous() or t.get_device() != k.get_device():
                raise TypeError(f"Kv4Cache: {n} must be a contiguous uint8 CUDA tensor on k's "
                                "device")
        raise ValueError("Kv4Cache: k and v must be [b, Hkv, L, d/2], the scales [b, Hkv, L, "
                         f"d/16], d 64 or 128, no dimension above 2^30; not {tuple(k.shape)}, "
                         f"{tuple(k_scale.shape)}, {tuple(v.shape)}, {tuple(v_scale.shape)}")

    @classmethod
    def empty(cls, batch, n_kv_heads, seq_len, head_dim=128, device="cuda"):
        codes = (batch, n_kv_heads, seq_len, head_dim // 2)
        scales = (batch, n_kv_heads, seq_len, head_dim // 16)
        return cls(*(torch.zeros(s, dtype=torch.uint8, device=device)
                     for s in (codes, scales, codes, scales)))


class Model:
    """A model recorded in the library (fdl_model_create): the description and
    the device pointers of the weights, which the caller keeps alive.
    `layers` holds per layer the tensors attn_norm, w_qkv, bias (or None), wo,
    ffn_norm, w_gu, wd."""

    def __init__(self, *, vocab, hidden, n_q_heads, n_kv_heads, ffn, mask_id, embed,
                 final_norm, lm_head, layers, head_dim=128, rope_theta=10000.0, rms_eps=1e-5):
        L = load()
        self._keep = (embed, final_norm, lm_head, layers)
        self.desc = ModelDesc(vocab, hidden, len(layers), n_q_heads, n_kv_heads, head_dim, ffn,
                              mask_id, rope_theta, rms_eps)
        arr = (LayerWeights * len(layers))()
        for k, Lw in enumerate(layers):
            arr[k] = LayerWeights(Lw["attn_norm"].data_ptr(), Lw["w_qkv"].data_ptr(),
                                  Lw["bias"].data_ptr() if Lw.get("bias") is not None else None,
                                  Lw["wo"].data_ptr(), Lw["ffn_norm"].data_ptr(),
                                  Lw["w_gu"].data_ptr(), Lw["wd"].data_ptr())
        w = ModelWeights(embed.data_ptr(), final_norm.data_ptr(), lm_head.data_ptr(), arr)
        h = ctypes.c_void_p()
        _check(L.fdl_model_create(ctypes.byref(self.desc), ctypes.byref(w), ctypes.byref(h)))
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            load().fdl_model_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Context:
    """One library context on one CUDA device. Holds a torch-allocated scratch
    buffer that grows to the largest workspace asked for."""

    def __init__(self, device: int | None = None):
        L = load()
        self.device = torch.cuda.current_device() if device is None else int(device)
        h = ctypes.c_void_p()
        _check(L.fdl_create(ctypes.byref(h), self.device))
        self._h = h
        self._ws = None
        self._seeds = {}        # empty tensors by dtype, from which others are made: an
                                # allocation without a dtype to read takes 1.4 us, not 2
        self._kv4_descs = {}    # descriptors by their values: a reference for the calls, scratch

    def close(self):
        if getattr(self, "_h", None):
            load().fdl_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- scratch ---------------------------------------------------------
    def workspace(self, nbytes: int) -> torch.Tensor:
        nbytes = max(int(nbytes), 16)
        if self._ws is None or self._ws.numel() < nbytes:
            self._ws = torch.empty(nbytes, dtype=torch.uint8, device=f"cuda:{self.device}")
        return self._ws

    def set_wait_timeout(self, ns: int):
        """Limit (ns) of the kernels' progress waits on this context
        (fdl_set_wait_timeout)."""
        _check(load().fdl_set_wait_timeout(self._h, int(ns)))

    def device_status(self, stream=None) -> int:
        """Synchronise and raise FdlError if a kernel recorded a device error."""
        _check(load().fdl_get_device_status(self._h, _stream(stream)))
        return FDL_OK

    # -- (a) attention ----------------------------------------------------
    def attn_desc(self, q, k_cache, block_start, scale=0.0) -> AttnDesc:
        b, B, Hq, d = q.shape
        _, Hkv, L, _ = k_cache.shape
        return AttnDesc(b, Hq, Hkv, d, L, int(block_start), B, _dtype_code(q), float(scale))

    def attention_workspace_bytes(self, desc: AttnDesc) -> int:
        return int(load().fdl_attention_workspace_bytes(self._h, ctypes.byref(desc)))

    def dualcache_attention(self, q, k_cache, v_cache, block_start, *, out=None, lse=None,
                            want_lse=False, scale=0.0, ws=None, stream=None):
        for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
            _need(t, n, q.dtype, 4)
        d = self.attn_desc(q, k_cache, block_start, scale)
        if out is None:
            out = torch.empty_like(q)
        if lse is None and want_lse:
            lse = torch.empty((d.batch, d.n_q_heads, d.block_len), dtype=torch.float32,
                              device=q.device)
        need = self.attention_workspace_bytes(d)
        if ws is None:
            ws = self.workspace(need)
        _check(load().fdl_dualcache_attention(self._h, ctypes.byref(d), _ptr(q), _ptr(k_cache),
                                              _ptr(v_cache), _ptr(out), _ptr(lse), _ptr(ws),
                                              ws.numel() * ws.element_size(), _stream(stream)))
        return (out, lse) if (want_lse or lse is not None) else out

    def kv_store(self, k_new, v_new, k_cache, v_cache, start, stream=None):
        _need(k_new, "k_new", k_cache.dtype, 4)
        _need(v_new, "v_new", k_cache.dtype, 4)
        _need(k_cache, "k_cache", None, 4)
        _need(v_cache, "v_cache", k_cache.dtype, 4)
        b, Hkv, L, d = k_cache.shape
        n = _i32(k_new.shape[1], "n")
        desc = AttnDesc(b, Hkv, Hkv, d, L, 0, 1, _dtype_code(k_cache), 0.0)
        _check(load().fdl_kv_store(self._h, ctypes.byref(desc), _ptr(k_new), _ptr(v_new),
                                   int(start), int(n), _ptr(k_cache), _ptr(v_cache),
                                   _stream(stream)))

    # -- 4-bit K/V cache ----------------------------------------------------
    # These calls are short on the GPU, so their host side is kept short too: one
    # test of everything that is usually right, and the words only when it is not.
    def _here(self, t, name, dtype, shape):
        """Raise unless t is a contiguous `dtype` tensor of `shape` on this device."""
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.get_device() != self.device:
            raise ValueError(f"{name} is on {t.device}, the context on cuda:{self.device}")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")

    def _on(self, stream):
        """Calls inside go to `stream`, and the tensors allocated for them belong to it."""
        if stream.device_index != self.device:
            raise ValueError(f"the stream is on cuda:{stream.device_index}, the context on "
                             f"cuda:{self.device}")
        return torch.cuda.stream(stream)

    def _seed(self, dtype):
        t = self._seeds.get(dtype)
        if t is None:
            t = self._seeds[dtype] = torch.empty(0, dtype=dtype, device=f"cuda:{self.device}")
        return t

    def _other_device(self, cache):
        raise ValueError(f"the cache is on cuda:{cache.device_index}, the context on "
                         f"cuda:{self.device}")

    def _kv4_rows(self, cache, k, v, n):
        """Descriptor of unquantised rows k, v (either may be None) [b, n, Hkv, d]."""
        one = k if k is not None else v
        b, h, d = cache.batch, cache.n_kv_heads, cache.head_dim
        try:
            strides, dtype = one.stride(), one.dtype
            s0, s1, s2, s3 = strides
            right = (s3 == 1 and one.shape == (b, n, h, d) and one.get_device() == self.device
                     and (one is v or v is None
                          or (v.stride() == strides and v.dtype is dtype and v.shape == one.shape
                              and v.get_device() == self.device))
                     and (dtype is torch.bfloat16 or dtype is torch.float32))
        except (AttributeError, ValueError):
            right = False
        if not right:
            self._refuse_rows(k, v, (b, n, h, d))
        # a dimension of one position has no stride of its own
        if b == 1 or n == 1 or h == 1:
            s0, s1, s2 = (s0 if b > 1 else n * h * d, s1 if n > 1 else h * d, s2 if h > 1 else d)
        if not (s0 or s1 or s2):
            raise ValueError("rows without any stride are not supported")
        return Kv4RowsDesc(b, h, d, cache.seq_len, FDL_BF16 if dtype is torch.bfloat16 else FDL_F32,
                           s0, s1, s2)

    def _refuse_rows(self, k, v, want):
        one = k if k is not None else v
        for t, name in ((k, "k"), (v, "v")):
            if t is None:
                continue
            if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype is not one.dtype:
                raise TypeError(f"{name} rows must be a CUDA tensor, k's and v's of one dtype")
            if t.get_device() != self.device:
                raise ValueError(f"{name} rows are on {t.device}, the context on "
                                 f"cuda:{self.device}")
            if t.shape != want:
                raise ValueError(f"{name} rows have shape {tuple(t.shape)}, not {want}")
            if t.stride(3) != 1:
                raise ValueError(f"{name} rows must be contiguous along head_dim")
        _dtype_code(one)
        raise ValueError("k and v rows must have the same strides")

    def kv4_store(self, k_new, v_new, cache: Kv4Cache, start, stream=None):
        """Quantise rows k_new, v_new [b, n, Hkv, d] (bf16 or f32; any strides with head_dim
        contiguous, the same for both) into positions [start, start + n) of the cache."""
        if stream is not None:
            with self._on(stream):
                return self.kv4_store(k_new, v_new, cache, start)
        if cache.device_index != self.device:
            self._other_device(cache)
        if not isinstance(k_new, torch.Tensor) or k_new.dim() != 4 or v_new is None:
            raise ValueError("kv4_store: k_new and v_new must be [b, n, Hkv, d]")
        n = _i32(k_new.shape[1], "n")
        d = self._kv4_rows(cache, k_new, v_new, n)
        rc = (_lib or load()).fdl_kv4_store(self._h, ctypes.byref(d), k_new.data_ptr(),
                                            v_new.data_ptr(), _i32(start, "start"), n,
                                            ctypes.byref(cache.buffers), _raw_stream(self.device))
        if rc:
            _check(rc)

    def kv4_load(self, cache: Kv4Cache, start=0, n=None, *, dtype=torch.bfloat16, k_out=None,
                 v_out=None, stream=None):
        """The values positions [start, start + n) of the cache stand for (n: to the end):
        (k, v) [b, n, Hkv, d], new tensors of `dtype` (bf16 or f32) or the given k_out and
        v_out (of one of them alone, only that one is read)."""
        if stream is not None:
            with self._on(stream):
                return self.kv4_load(cache, start, n, dtype=dtype, k_out=k_out, v_out=v_out)
        if cache.device_index != self.device:
            self._other_device(cache)
        start = _i32(start, "start")
        n = cache.seq_len - start if n is None else _i32(n, "n")
        if k_out is None and v_out is None:
            if n < 1:
                raise ValueError(f"kv4_load: {n} rows")
            b, h, hd = cache.batch, cache.n_kv_heads, cache.head_dim
            if dtype is not torch.bfloat16 and dtype is not torch.float32:
                raise TypeError(f"unsupported dtype {dtype}")
            if n > cache.seq_len:
                raise ValueError(f"kv4_load: {n} rows of {cache.seq_len}")
            k_out = self._seed(dtype).new_empty(b, n, h, hd)
            v_out = torch.empty_like(k_out)
            d = Kv4RowsDesc(b, h, hd, cache.seq_len,
                            FDL_BF16 if dtype is torch.bfloat16 else FDL_F32, 0, 0, 0)
        else:
            d = self._kv4_rows(cache, k_out, v_out, n)
        rc = (_lib or load()).fdl_kv4_load(
            self._h, ctypes.byref(d), ctypes.byref(cache.buffers), start, n,
            None if k_out is None else k_out.data_ptr(),
            None if v_out is None else v_out.data_ptr(), _raw_stream(self.device))
        if rc:
            _check(rc)
        return k_out, v_out

    def kv4_attn_desc(self, q, cache: Kv4Cache, block_start, window=(-1, -1), sinks=0,
                      scale=0.0) -> Kv4AttnDesc:
        b, B, Hq, d = q.shape
        if b != cache.batch or d != cache.head_dim:
            raise ValueError(f"q {tuple(q.shape)} does not fit a cache of {cache.batch} sequences "
                             f"and head_dim {cache.head_dim}")
        left, right = window
        return Kv4AttnDesc(b, _i32(Hq, "q heads"), cache.n_kv_heads, d, cache.seq_len,
                           _i32(block_start, "block_start"), _i32(B, "block length"), FDL_BF16,
                           float(scale), _i32(left, "window"), _i32(right, "window"),
                           _i32(sinks, "sinks"))

    def kv4_attention_workspace_bytes(self, desc: Kv4AttnDesc) -> int:
        return int(load().fdl_kv4_attention_workspace_bytes(self._h, ctypes.byref(desc)))

    def kv4_attention_plan(self, desc: Kv4AttnDesc) -> Kv4Plan:
        plan = Kv4Plan()
        _check(load().fdl_kv4_attention_plan(self._h, ctypes.byref(desc), ctypes.byref(plan)))
        return plan

    def kv4_attention(self, q, cache: Kv4Cache, block_start, *, kv_len=None, window=(-1, -1),
                      sinks=0, out=None, lse=None, want_lse=False, scale=0.0, ws=None,
                      stream=None):
        """Block attention over a 4-bit cache (fdl_kv4_attention). q [b, B, Hq, d] bf16, the
        block's rows being in the cache already (kv4_store). kv_len [b] int32 (CUDA): valid
        positions of each sequence; window (left, right): positions around the block that it
        sees, -1 for all; sinks: first positions that stay visible. Without ws the scratch is
        allocated for the call, so calls on several streams, and captured ones, do not share it."""
        if stream is not None:
            with self._on(stream):
                return self.kv4_attention(q, cache, block_start, kv_len=kv_len, window=window,
                                          sinks=sinks, out=out, lse=lse, want_lse=want_lse,
                                          scale=scale, ws=ws)
        if cache.device_index != self.device:
            self._other_device(cache)
        if not isinstance(q, torch.Tensor) or q.dim() != 4:
            raise ValueError("kv4_attention: q must be [b, B, Hq, d]")
        if q.get_device() != self.device or q.dtype is not torch.bfloat16 \
                or not q.is_contiguous():
            self._here(q, "q", torch.bfloat16, q.shape)
        b, B, Hq, hd = q.shape
        # numbers before they become a key: a tensor would be one by its identity, whatever
        # it holds by the next call
        left, right = window
        left, right, sinks, scale = int(left), int(right), int(sinks), float(scale)
        block_start = int(block_start)
        key = (b, B, Hq, hd, cache.batch, cache.n_kv_heads, cache.seq_len, cache.head_dim,
               block_start, left, right, sinks, scale)
        known = self._kv4_descs.get(key)
        if known is None:
            if len(self._kv4_descs) >= 4096:
                self._kv4_descs.clear()
            d = self.kv4_attn_desc(q, cache, block_start, (left, right), sinks, scale)
            known = self._kv4_descs[key] = ctypes.byref(d), self.kv4_attention_workspace_bytes(d)
        d, need = known
        if kv_len is not None:
            self._here(kv_len, "kv_len", torch.int32, (b,))
        if out is None:
            out = torch.empty_like(q)
        else:
            self._here(out, "out", torch.bfloat16, q.shape)
        if lse is not None:
            self._here(lse, "lse", torch.float32, (b, Hq, B))
        elif want_lse:
            lse = self._seed(torch.float32).new_empty(b, Hq, B)
        if ws is not None:
            self._here(ws, "ws", ws.dtype, ws.shape)
        elif need > 16:                      # most shapes need none
            ws = self._seed(torch.uint8).new_empty(need)
        rc = (_lib or load()).fdl_kv4_attention(
            self._h, d, q.data_ptr(), ctypes.byref(cache.buffers),
            None if kv_len is None else kv_len.data_ptr(), out.data_ptr(),
            None if lse is None else lse.data_ptr(), None if ws is None else ws.data_ptr(),
            0 if ws is None else ws.numel() * ws.element_size(), _raw_stream(self.device))
        if rc:
            _check(rc)
        return (out, lse) if (want_lse or lse is not None) else out

    # -- (b) LM head + confidence ----------------------------------------
    def lmhead_workspace_bytes(self, desc: LMHeadDesc) -> int:
        return int(load().fdl_lmhead_workspace_bytes(self._h, ctypes.byref(desc)))

    def lmhead_confidence(self, h, w, bias_tok=None, bias_val=None, *, conf=None, tok=None,
                          ws=None, stream=None):
        _need(h, "h", None, 2)
        _need(w, "w", h.dtype, 2)
        if bias_tok is not None:
            _need(bias_tok, "bias_tok", torch.int32, 1)
            _need(bias_val, "bias_val", torch.float32, 1)
        M, D = h.shape
        V = w.shape[0]
        d = LMHeadDesc(M, D, V, _dtype_code(h))
        if conf is None:
            conf = torch.empty(M, dtype=torch.float32, device=h.device)
        if tok is None:
            tok = torch.empty(M, dtype=torch.int32, device=h.device)
        if ws is None:
            ws = self.workspace(self.lmhead_workspace_bytes(d))
        _check(load().fdl_lmhead_confidence(self._h, ctypes.byref(d), _ptr(h), _ptr(w),
                                            _ptr(bias_tok), _ptr(bias_val), _ptr(conf),
                                            _ptr(tok), _ptr(ws), ws.numel() * ws.element_size(),
                                            _stream(stream)))
        return conf, tok

    def lmhead_confidence_noalloc(self, h, w, bias_tok=None, bias_val=None, *, conf=None,
                                  tok=None, stream=None):
        """fdl_lmhead_confidence_noalloc: no workspace argument; the library's
        built-in 8 MiB scratch array is used (see include/fdllm.h)."""
        _need(h, "h", None, 2)
        _need(w, "w", h.dtype, 2)
        if bias_tok is not None:
            _need(bias_tok, "bias_tok", torch.int32, 1)
            _need(bias_val, "bias_val", torch.float32, 1)
        M, D = h.shape
        d = LMHeadDesc(M, D, w.shape[0], _dtype_code(h))
        if conf is None:
            conf = torch.empty(M, dtype=torch.float32, device=h.device)
        if tok is None:
            tok = torch.empty(M, dtype=torch.int32, device=h.device)
        _check(load().fdl_lmhead_confidence_noalloc(self._h, ctypes.byref(d), _ptr(h), _ptr(w),
                                                    _ptr(bias_tok), _ptr(bias_val), _ptr(conf),
                                                    _ptr(tok), _stream(stream)))
        return conf, tok

    # -- (b) threshold select + scatter -----------------------------------
    def threshold_unmask(self, conf, tok, x, masked, block_start, tau, *, remaining=None,
                         n_decoded=None, stream=None):
        _need(conf, "conf", torch.float32, 2)
        _need(tok, "tok", torch.int32, 2)
        _need(x, "x", torch.int32, 2)
        _need(masked, "masked", torch.uint8, 2)
        b, L = x.shape
        B = conf.shape[1]
        if remaining is None:
            remaining = torch.empty(b, dtype=torch.int32, device=x.device)
        d = UnmaskDesc(b, L, int(block_start), B, float(tau))
        _check(load().fdl_threshold_unmask(self._h, ctypes.byref(d), _ptr(conf), _ptr(tok),
                                           _ptr(x), _ptr(masked), _ptr(remaining),
                                           _ptr(n_decoded), _stream(stream)))
        return remaining

    # -- transformer scaffold ------------------------------------------------
    def rmsnorm(self, h, weight, eps, *, out=None, row_map=None, rows=None, stream=None):
        """bf16 RMSNorm of f32 rows of h (optionally gathered through row_map)."""
        _need(h, "h", torch.float32, 2)
        _need(weight, "weight", torch.float32, 1)
        n = rows if rows is not None else (row_map.numel() if row_map is not None else h.shape[0])
        if out is None:
            out = torch.empty((n, h.shape[1]), dtype=torch.bfloat16, device=h.device)
        _check(load().fdl_rmsnorm(self._h, int(n), h.shape[1], _ptr(h), _ptr(row_map),
                                  _ptr(weight), float(eps), _ptr(out), _stream(stream)))
        return out

    def embed(self, ids, table, *, out=None, row_map=None, stream=None):
        """f32 rows of the embedding table: table[ids[row_map[i]]] (or ids[i])."""
        _need(ids, "ids", torch.int32, None)
        _need(table, "table", torch.bfloat16, 2)
        n = row_map.numel() if row_map is not None else ids.numel()
        if out is None:
            out = torch.empty((n, table.shape[1]), dtype=torch.float32, device=ids.device)
        _check(load().fdl_embed(self._h, int(n), table.shape[1], _ptr(ids), _ptr(row_map),
                                _ptr(table), _ptr(out), _stream(stream)))
        return out

    def qkv_rope_store(self, x, w, rope, q_out, k_cache, v_cache, *, n_q_heads, rows_per_seq,
                       pos0, bias=None, stream=None):
        """[q|k|v] = x w^T (+bias), RoPE on q and k, q -> q_out, k/v -> caches."""
        _need(x, "x", torch.bfloat16, 2)
        _need(w, "w", torch.bfloat16, 2)
        b, hkv, L, d = k_cache.shape
        d_ = QKVDesc(x.shape[0], x.shape[1], int(n_q_heads), hkv, d, b, L, int(rows_per_seq),
                     int(pos0), rope.shape[0])
        _check(load().fdl_qkv_rope_store(self._h, ctypes.byref(d_), _ptr(x), _ptr(w),
                                         _ptr(bias), _ptr(rope), _ptr(q_out), _ptr(k_cache),
                                         _ptr(v_cache), _stream(stream)))
        return q_out

    def qkv_attention(self, x, w, rope, q_out, k_cache, v_cache, out, *, n_q_heads,
                      rows_per_seq, pos0, bias=None, h=None, norm_w=None, eps=1e-5,
                      stream=None):
        """[x = RMSNorm(h) * norm_w if norm_w is given], qkv_rope_store of the block
        rows, then DualCache attention of the block [pos0, pos0 + rows_per_seq) of
        every sequence over the caches -> out."""
        _need(x, "x", torch.bfloat16, 2)
        _need(w, "w", torch.bfloat16, 2)
        if norm_w is not None:
            _need(h, "h", torch.float32, 2)
        b, hkv, L, d = k_cache.shape
        d_ = QKVDesc(x.shape[0], x.shape[1], int(n_q_heads), hkv, d, b, L, int(rows_per_seq),
                     int(pos0), rope.shape[0])
        _check(load().fdl_qkv_attention(self._h, ctypes.byref(d_), _ptr(h), _ptr(norm_w),
                                        float(eps), _ptr(x), _ptr(w), _ptr(bias), _ptr(rope),
                                        _ptr(q_out), _ptr(k_cache), _ptr(v_cache), _ptr(out),
                                        _stream(stream)))
        return out

    def generate(self, model: Model, prompt, gen_len, *, block=32, tau=0.9, cache="dual",
                 bias_tok=None, bias_val=None, device_loop=False, batching="lockstep",
                 kv="bf16", stream=None):
        """The whole decode in the library (fdl_generate). prompt [b, P] int32,
        a CUDA tensor or a host tensor (then copied to the device first, and
        the result copied back to a host tensor: the public call with host
        buffers). cache: "dual", "prefix" or "none"; bias_tok / bias_val [b,
        gen_len] (CUDA, int32 / float32): optional planted logit bias of the
        generated positions. device_loop: the decode as one CUDA graph with the
        steps sequenced on the device (kept in the context for the next call
        with the same arguments; the workspace is kept by this Context so that
        it does). batching (DualCache, host loop for the last two): "lockstep",
        "compact" (cached steps only on the sequences with masked positions
        left in the block) or "per_sequence" (each sequence moves to its next
        block on its own). kv: how the layers' K/V are held, "bf16" or "4bit"
        (DualCache or PrefixCache, lockstep). Returns (x [b, P + gen_len] int32, steps)."""
        on_host = not prompt.is_cuda
        dev = torch.device("cuda", self.device)
        if on_host:
            prompt = prompt.to(dev, non_blocking=True)
        _need(prompt, "prompt", torch.int32, 2)
        b, P = prompt.shape
        if bias_tok is not None:
            _need(bias_tok, "bias_tok", torch.int32, 2)
            _need(bias_val, "bias_val", torch.float32, 2)
        L = load()
        n = L.fdl_generate_workspace_bytes_kv(self._h, model._h, b, P + gen_len, int(block),
                                              KV_FORMATS[kv])
        if n == 0:
            raise ValueError("generate: bad shape")
        if getattr(self, "_gen_ws", None) is None or self._gen_ws.numel() < n:
            self._gen_ws = None
            self._gen_ws = torch.empty(n, dtype=torch.uint8, device=dev)
        ws = self._gen_ws
        x = torch.empty((b, P + gen_len), dtype=torch.int32, device=dev)
        steps = ctypes.c_int(0)
        opts = GenerateOpts(CACHE_MODES[cache], int(bool(device_loop)),
                            None if bias_tok is None else bias_tok.data_ptr(),
                            None if bias_val is None else bias_val.data_ptr(),
                            BATCHING[batching], KV_FORMATS[kv])
        _check(L.fdl_generate(self._h, model._h, _ptr(prompt), b, P, int(gen_len), int(block),
                              float(tau), ctypes.byref(opts), _ptr(x), ctypes.byref(steps),
                              _ptr(ws), ws.numel(), _stream(stream)))
        if on_host:
            x = x.cpu()
        return x, steps.value

    def linear_residual(self, x, w, h, *, stream=None):
        """h += x w^T (h f32)."""
        _need(x, "x", torch.bfloat16, 2)
        _need(w, "w", torch.bfloat16, 2)
        _need(h, "h", torch.float32, 2)
        _check(load().fdl_linear_residual(self._h, x.shape[0], w.shape[0], x.shape[1], _ptr(x),
                                          _ptr(w), _ptr(h), _stream(stream)))
        return h

    def linear_swiglu(self, x, w_gu, *, out=None, stream=None):
        """silu(x Wg^T) * (x Wu^T) with gate/up rows interleaved in w_gu."""
        _need(x, "x", torch.bfloat16, 2)
        _need(w_gu, "w_gu", torch.bfloat16, 2)
        F = w_gu.shape[0] // 2
        if out is None:
            out = torch.empty((x.shape[0], F), dtype=torch.bfloat16, device=x.device)
        _check(load().fdl_linear_swiglu(self._h, x.shape[0], F, x.shape[1], _ptr(x), _ptr(w_gu),
                                        _ptr(out), _stream(stream)))
        return out

    def ffn(self, x, w_gu, w_down, h, *, f=None, norm_w=None, eps=1e-5, stream=None):
        """[x = RMSNorm(h) * norm_w if norm_w is given], then
        h += (silu(x Wg^T) * (x Wu^T)) Wd^T; returns f, the SwiGLU output."""
        _need(x, "x", torch.bfloat16, 2)
        _need(w_gu, "w_gu", torch.bfloat16, 2)
        _need(w_down, "w_down", torch.bfloat16, 2)
        _need(h, "h", torch.float32, 2)
        rows, hidden = x.shape
        F = w_gu.shape[0] // 2
        if f is None:
            f = torch.empty((rows, F), dtype=torch.bfloat16, device=x.device)
        _check(load().fdl_ffn(self._h, rows, hidden, F, _ptr(norm_w), float(eps), _ptr(x),
                              _ptr(w_gu), _ptr(w_down), _ptr(f), _ptr(h), _stream(stream)))
        return f

    def full_attention(self, q, k_cache, v_cache, *, q_start=0, out=None, scale=0.0,
                       stream=None):
        """Bidirectional attention of the positions [q_start, L) over all L
        positions of the caches: q, out [b, L - q_start, Hq, d] (q_start = 0:
        every position, the refresh; q_start = s: the block and the suffix of a
        PrefixCache step)."""
        _need(q, "q", torch.bfloat16, 4)
        _need(k_cache, "k_cache", torch.bfloat16, 4)
        _need(v_cache, "v_cache", torch.bfloat16, 4)
        b, nq, Hq, d = q.shape
        hkv, L = k_cache.shape[1], k_cache.shape[2]
        if nq != L - int(q_start):
            raise ValueError(f"full_attention: q has {nq} rows per sequence, the caches "
                             f"{L} - q_start {q_start}")
        desc = AttnDesc(b, Hq, hkv, d, L, int(q_start), nq, FDL_BF16, float(scale))
        if out is None:
            out = torch.empty_like(q)
        _check(load().fdl_full_attention(self._h, ctypes.byref(desc), _ptr(q), _ptr(k_cache),
                                         _ptr(v_cache), _ptr(out), _stream(stream)))
        return out

"""Thin ctypes binding of libkvq (include/kvq.h). Argument marshalling only: every step of
the computation runs in the library's CUDA kernels. PyTorch provides device memory and
streams. The binding fails loudly when the library is missing or a call returns an error;
there is no fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import re
from dataclasses import dataclass

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkvq.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "kvq.h")

KVQ_OK = 0
ERR_INVALID_ARG, ERR_CAPACITY, ERR_UNSUPPORTED, ERR_CUDA, ERR_WORKSPACE, ERR_TIMEOUT = 1, 2, 3, 4, 5, 6
STATUS = {0: "KVQ_OK", 1: "KVQ_ERR_INVALID_ARG", 2: "KVQ_ERR_CAPACITY", 3: "KVQ_ERR_UNSUPPORTED",
          4: "KVQ_ERR_CUDA", 5: "KVQ_ERR_WORKSPACE", 6: "KVQ_ERR_TIMEOUT"}
FMT_LOOPVQ, FMT_KIVI = 0, 1
OUT_BF16, OUT_FP32 = 0, 1
PER_CHANNEL, PER_TOKEN = 0, 1
DT_BF16, DT_FP32, DT_FP16 = 0, 1, 2
SLOT_KEEP, SLOT_FREE = -1, -2
FORK_MAX = 256
PAGE = 8


class KvqError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}: {detail}")


class VqCfg(ctypes.Structure):
    _fields_ = [("D", ctypes.c_int), ("T", ctypes.c_int), ("Tc", ctypes.c_int), ("G", ctypes.c_int),
                ("K", ctypes.c_int), ("n_layers", ctypes.c_int), ("n_heads", ctypes.c_int),
                ("sink", ctypes.c_int), ("recent", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("max_batch", ctypes.c_int), ("max_ctx", ctypes.c_int), ("rope_base", ctypes.c_float)]


class VqCacheC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("idx_k", "idx_v", "win_k", "win_v", "bt_k", "bt_v", "cb_k", "cb_v",
                 "rope_cos", "rope_sin", "seq_len", "n_pages", "cbp_k", "cbp_v")]


class VqSizes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("idx", "win", "bt", "bt_v", "cb", "rope", "per_request", "cbp")]


class KiviCfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in
                ("D", "n_heads", "n_q_heads", "k_bits", "v_bits", "group", "residual", "max_batch",
                 "max_tokens")]


KIVI_CACHE_FIELDS = ("k_codes", "k_scale", "k_zero", "v_codes", "v_scale", "v_zero",
                     "k_resid", "v_resid", "n_tok", "n_quant_k", "n_quant_v", "sync")


class KiviCacheC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in KIVI_CACHE_FIELDS]


class Rows(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_t", ctypes.c_int64),
                ("stride_h", ctypes.c_int64), ("heads", ctypes.c_int), ("dtype", ctypes.c_int)]


class Dist(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_t", ctypes.c_int64),
                ("dtype", ctypes.c_int)]


_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_SIGS = {
    "kvq_version": (_I, []),
    "kvq_status_string": (ctypes.c_char_p, [_I]),
    "kvq_last_error": (ctypes.c_char_p, []),
    "kvq_device_error": (_I, []),
    "kvq_vq_cache_sizes": (_I, [_P, _P]),
    "kvq_rope_table": (_I, [_P, _P, _P, _P]),
    "kvq_slice_codebooks": (_I, [_P, _P, _P, _P]),
    "kvq_slice_codebooks_fp16": (_I, [_P, _P, _P, _P]),
    "kvq_split_codebooks": (_I, [_P, _P, _P, _P]),
    "kvq_encode_vq": (_I, [_P, _P, _I64, _I64, _I64, _I, _I, _I, _P, _P, _I, _I, _I, _P, _P]),
    "kvq_prefill_vq": (_I, [_P, _P, _I, _P, _P, _I64, _I64, _I64, _I, _I, _I, _P, _P]),
    "kvq_append_page": (_I, [_P, _P, _I, _I, _P, _P, _I, _P]),
    "kvq_quantize_kivi": (_I, [_P, _I, _P, _I64, _I64, _I, _I, _P, _P, _P, _I, _P]),
    "kvq_kivi_prefill": (_I, [_P, _P, _P, _P, _I64, _I64, _I, _I, _I, _P]),
    "kvq_kivi_append": (_I, [_P, _P, _P, _P, _I, _P]),
    "kvq_kivi_commit": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _P]),
    "kvq_kivi_read": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _I, _I64, _I64, _P]),
    "kvq_qk_norm_rope": (_I, [_I, _I, _I, _P, _P, _P, _P, _P, _F, _P, _P, _I, _P, _P, _P, _P, _P]),
    "kvq_kivi_tree_attn": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _P, _I, _P, _SZ, _P]),
    "kvq_kivi_tree_workspace_size": (_SZ, [_P, _I, _I]),
    "kvq_kivi_prefix_attn": (_I, [_P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _P, _I, _P, _SZ, _P]),
    "kvq_kivi_prefix_workspace_size": (_SZ, [_P, _P, _I, _I]),
    "kvq_cache_fork": (_I, [_I, _P, _P, _P, _P, _P, _I, _I, _P]),
    "kvq_verify_draft": (_I, [_I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "kvq_decode_attn": (_I, [_I, _P, _P, _I, _I, _P, _I, _P, _I, _I, _P, _SZ, _P]),
    "kvq_decode_attn_noalloc": (_I, [_I, _P, _P, _I, _I, _P, _I, _P, _I, _I, _P]),
    "kvq_decode_workspace_size": (_SZ, [_I, _P, _I, _I]),
    "kvq_decode_auto_splits": (_I, [_I, _P, _I]),
}

_lib = None


def header_functions() -> list[str]:
    """Names of the functions include/kvq.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(kvq_[a-z0-9_]+)\s*\(", text)))


def lib() -> ctypes.CDLL:
    """The loaded libkvq.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libkvq.so not found at {LIB_PATH}: run __graft_entry__.build() "
                               "(or python sub_bit_quantized_gb300/_build.py) first")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _on(stream, device):
    """Context in which PyTorch allocates and fills on ``stream`` (None: the current one). A block that it frees again
    then waits for what is queued there, and one that it gives out has nothing pending elsewhere."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        h = _stream(stream)
        stream = torch.cuda.ExternalStream(h, device=device) if h else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _check(st: int, where: str):
    if st != KVQ_OK:
        raise KvqError(st, where, lib().kvq_last_error().decode())


def version() -> int:
    return lib().kvq_version()


def device_error() -> int:
    """Read and clear the device error word (synchronizes the device)."""
    return lib().kvq_device_error()


def _bits(t: torch.Tensor, dtypes) -> torch.Tensor:
    if t.dtype not in dtypes:
        raise TypeError(f"expected one of {dtypes}, got {t.dtype}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("expected a contiguous CUDA tensor")
    return t


_DT = {torch.bfloat16: DT_BF16, torch.float32: DT_FP32, torch.float16: DT_FP16}


def _operand(name: str, t: torch.Tensor, dtypes, shape, contiguous: bool = True) -> torch.Tensor:
    """``t`` if it has one of the types, the shape (None: any size) and lies on the current device."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: expected one of {dtypes}, got {t.dtype}")
    if t.dim() != len(shape) or any(s is not None and s != n for s, n in zip(shape, t.shape)):
        raise ValueError(f"{name}: expected the shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name}: expected a tensor on the current CUDA device, got one on {t.device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t


def _step(t: torch.Tensor, dim: int) -> int:
    """The stride of a dimension, 0 where it has one entry (any number may stand there)."""
    return t.stride(dim) if t.shape[dim] > 1 else 0


class _Call:
    """Pre-marshalled arguments of a repeated library call. It holds its tensors, and runs on ``stream``
    or else on the stream that is current when it is called."""

    def __init__(self, name: str, stream, device, keep):
        self._name = name
        self._stream = None if stream is None else _stream(stream)
        self._device, self._keep = device.index, (stream, keep)

    def _bind(self, *args):
        """All arguments but the stream, converted to their C types once: the call itself then goes through a
        prototype without conversions (2.2 -> 1.2 us of host time for 17 arguments)."""
        f = getattr(lib(), self._name)
        self._args = [x if x is None or hasattr(x, "_obj") else t(x) for x, t in zip(args, f.argtypes)]
        self._f = lib()[self._name]

    def __call__(self):
        if torch._C._cuda_getDevice() != self._device:
            raise ValueError(f"{self._name}: its tensors are on device {self._device}, not on the current one")
        s = self._stream
        if s is None:
            s = torch._C._cuda_getCurrentRawStream(self._device)
        st = self._f(*self._args, ctypes.c_void_p(s))
        if st != KVQ_OK:
            _check(st, self._name)


# ------------------------------------------------------------------------------------------
# LoopVQ
# ------------------------------------------------------------------------------------------

@dataclass
class VqConfig:
    D: int = 128
    T: int = 4
    Tc: int = 2
    G: int = 16
    K: int = 256
    n_layers: int = 1
    n_heads: int = 1
    sink: int = 8
    recent: int = 64
    max_pages: int = 0
    max_batch: int = 1
    max_ctx: int = 2
    rope_base: float = 1.0e4

    @property
    def NB(self) -> int:
        return self.T // self.Tc

    @property
    def c(self) -> int:
        return self.G // self.Tc

    @property
    def NG(self) -> int:
        return self.D // self.c

    @property
    def win_slots(self) -> int:
        return self.sink + self.recent + PAGE

    def to_c(self) -> VqCfg:
        return VqCfg(self.D, self.T, self.Tc, self.G, self.K, self.n_layers, self.n_heads, self.sink,
                     self.recent, self.max_pages, self.max_batch, self.max_ctx, float(self.rope_base))


class VqCache:
    """A LoopVQ cache whose buffers PyTorch allocates on the current device.

    Shapes follow include/kvq.h. ``cb_k`` / ``cb_v`` hold the full codebooks; call
    ``load_codebooks`` to set them (it also cuts the per-step slices on the GPU), and
    ``rope_table`` is filled on construction.
    """

    def __init__(self, cfg: VqConfig, device="cuda"):
        self.cfg = cfg
        c = cfg
        dev = torch.device(device)
        L, NB, B, H, P = c.n_layers, c.NB, c.max_batch, c.n_heads, c.max_pages
        self.idx_k = torch.zeros((L, NB, B, H, P, PAGE * c.NG), dtype=torch.uint8, device=dev)
        self.idx_v = torch.zeros_like(self.idx_k)
        self.win_k = torch.zeros((L, c.T, B, H, c.win_slots, c.D), dtype=torch.bfloat16, device=dev)
        self.win_v = torch.zeros_like(self.win_k)
        self.bt_k = torch.zeros((L, c.T, H, 2, c.K, c.D // 2), dtype=torch.float32, device=dev)
        self.bt_v = torch.zeros((L, c.T, H, c.K, c.D), dtype=torch.float16, device=dev)
        self.cb_k = torch.zeros((L, NB, H, c.NG, c.K, c.G), dtype=torch.float32, device=dev)
        self.cb_v = torch.zeros_like(self.cb_k)
        sizes = vq_cache_sizes(cfg)
        # codebook parts for the tensor-core page roll (kvq_split_codebooks)
        self.cbp_k = torch.zeros(sizes.cbp, dtype=torch.uint8, device=dev)
        self.cbp_v = torch.zeros_like(self.cbp_k)
        self.rope_cos = torch.empty((c.max_ctx, c.D // 2), dtype=torch.float32, device=dev)
        self.rope_sin = torch.empty_like(self.rope_cos)
        self.seq_len = torch.zeros(B, dtype=torch.int32, device=dev)
        self.n_pages = torch.zeros(B, dtype=torch.int32, device=dev)
        self._cfg_c = cfg.to_c()
        sizes = vq_cache_sizes(cfg)
        assert sizes.idx == self.idx_k.numel() and sizes.win == self.win_k.numel() * 2
        assert sizes.bt == self.bt_k.numel() * 4 and sizes.bt_v == self.bt_v.numel() * 2
        assert sizes.cb == self.cb_k.numel() * 4
        kvq_rope_table(cfg, self.rope_cos, self.rope_sin)

    def c_struct(self) -> VqCacheC:
        return VqCacheC(*[_ptr(getattr(self, n)) for n in
                          ("idx_k", "idx_v", "win_k", "win_v", "bt_k", "bt_v", "cb_k", "cb_v",
                           "rope_cos", "rope_sin", "seq_len", "n_pages", "cbp_k", "cbp_v")])

    def load_codebooks(self, cb_k: torch.Tensor, cb_v: torch.Tensor, stream=None):
        self.cb_k.copy_(cb_k)
        self.cb_v.copy_(cb_v)
        kvq_slice_codebooks(self.cfg, self.cb_k, self.bt_k, stream)
        kvq_slice_codebooks_fp16(self.cfg, self.cb_v, self.bt_v, stream)
        kvq_split_codebooks(self.cfg, self.cb_k, self.cbp_k, stream)
        kvq_split_codebooks(self.cfg, self.cb_v, self.cbp_v, stream)


def vq_cache_sizes(cfg: VqConfig) -> VqSizes:
    out = VqSizes()
    c = cfg.to_c()
    _check(lib().kvq_vq_cache_sizes(ctypes.byref(c), ctypes.byref(out)), "kvq_vq_cache_sizes")
    return out


def kvq_rope_table(cfg: VqConfig, rope_cos, rope_sin, stream=None):
    c = cfg.to_c()
    _check(lib().kvq_rope_table(ctypes.byref(c), _ptr(rope_cos), _ptr(rope_sin), _stream(stream)),
           "kvq_rope_table")


def kvq_slice_codebooks(cfg: VqConfig, cb, bt, stream=None):
    c = cfg.to_c()
    _check(lib().kvq_slice_codebooks(ctypes.byref(c), _ptr(cb), _ptr(bt), _stream(stream)),
           "kvq_slice_codebooks")


def kvq_slice_codebooks_fp16(cfg: VqConfig, cb, bt16, stream=None):
    c = cfg.to_c()
    _check(lib().kvq_slice_codebooks_fp16(ctypes.byref(c), _ptr(cb), _ptr(bt16), _stream(stream)),
           "kvq_slice_codebooks_fp16")


def kvq_split_codebooks(cfg: VqConfig, cb, cbp, stream=None):
    c = cfg.to_c()
    _check(lib().kvq_split_codebooks(ctypes.byref(c), _ptr(cb), _ptr(cbp), _stream(stream)), "kvq_split_codebooks")


def kvq_encode_vq(cfg: VqConfig, x, x_strides, seq_begin, n_seq, n_tok, cb, idx, page_begin=0,
                  g_begin=0, g_count=None, n_ties=None, stream=None):
    """x: bf16 tensor (or base pointer with explicit element strides (t, b, h))."""
    c = cfg.to_c()
    g_count = cfg.NG - g_begin if g_count is None else g_count
    st, sb, sh = x_strides
    _check(lib().kvq_encode_vq(ctypes.byref(c), _ptr(x), st, sb, sh, seq_begin, n_seq, n_tok,
                               _ptr(cb), _ptr(idx), page_begin, g_begin, g_count, _ptr(n_ties),
                               _stream(stream)), "kvq_encode_vq")


def kvq_prefill_vq(cfg: VqConfig, cache: VqCache, layer: int, xk, xv, seq_begin: int, L: int,
                   n_ties=None, stream=None):
    """xk, xv: bf16 [T][n_seq][H][L][D] pre-RoPE keys / values of one layer."""
    T, n_seq, H, Lx, D = xk.shape
    assert xv.shape == xk.shape and Lx >= L
    _bits(xk, (torch.bfloat16,))
    _bits(xv, (torch.bfloat16,))
    c = cfg.to_c()
    kc = cache.c_struct()
    st, sb, sh = n_seq * H * Lx * D, H * Lx * D, Lx * D
    _check(lib().kvq_prefill_vq(ctypes.byref(c), ctypes.byref(kc), layer, _ptr(xk), _ptr(xv), st, sb, sh,
                                seq_begin, n_seq, L, _ptr(n_ties), _stream(stream)), "kvq_prefill_vq")


def kvq_append_page(cfg: VqConfig, cache: VqCache, layer: int, loop_step: int, k_new, v_new,
                    stream=None):
    """k_new, v_new: bf16 [n_seq][H][D] pre-RoPE key / value of the newest token at (layer, step)."""
    _bits(k_new, (torch.bfloat16,))
    _bits(v_new, (torch.bfloat16,))
    c = cfg.to_c()
    kc = cache.c_struct()
    _check(lib().kvq_append_page(ctypes.byref(c), ctypes.byref(kc), layer, loop_step, _ptr(k_new),
                                 _ptr(v_new), k_new.shape[0], _stream(stream)), "kvq_append_page")


# ------------------------------------------------------------------------------------------
# KIVI
# ------------------------------------------------------------------------------------------

@dataclass
class KiviConfig:
    """kvq_kivi_cfg. n_q_heads defaults to n_heads (multi-head attention)."""
    D: int = 128
    n_heads: int = 1
    n_q_heads: int | None = None
    k_bits: int = 2
    v_bits: int = 2
    group: int = 32
    residual: int = 128
    max_batch: int = 1
    max_tokens: int = 0

    @property
    def q_heads(self) -> int:
        return self.n_heads if self.n_q_heads is None else self.n_q_heads

    def to_c(self) -> KiviCfg:
        return KiviCfg(self.D, self.n_heads, self.q_heads, self.k_bits, self.v_bits, self.group,
                       self.residual, self.max_batch, self.max_tokens)


class KiviCache:
    """Device buffers of a KIVI cache (layouts of kvq_kivi_cache), zero-filled."""

    def __init__(self, cfg: KiviConfig, device="cuda"):
        self.cfg = cfg
        c = cfg
        dev = torch.device(device)
        B, H, N, D, Gq = c.max_batch, c.n_heads, c.max_tokens, c.D, c.group
        self.k_codes = torch.zeros((B, H, N, D * c.k_bits // 8), dtype=torch.uint8, device=dev)
        self.v_codes = torch.zeros((B, H, N, D * c.v_bits // 8), dtype=torch.uint8, device=dev)
        self.k_scale = torch.zeros((B, H, N // Gq, D), dtype=torch.float16, device=dev)
        self.k_zero = torch.zeros_like(self.k_scale)
        self.v_scale = torch.zeros((B, H, N, D // Gq), dtype=torch.float16, device=dev)
        self.v_zero = torch.zeros_like(self.v_scale)
        self.k_resid = torch.zeros((B, H, max(c.residual, 1), D), dtype=torch.float16, device=dev)
        self.v_resid = torch.zeros_like(self.k_resid)
        self.n_tok = torch.zeros(B, dtype=torch.int32, device=dev)
        self.n_quant_k = torch.zeros(B, dtype=torch.int32, device=dev)
        self.n_quant_v = torch.zeros(B, dtype=torch.int32, device=dev)
        self.sync = torch.zeros(B, dtype=torch.int32, device=dev)

    def c_struct(self) -> KiviCacheC:
        return KiviCacheC(*[_ptr(getattr(self, n)) for n in KIVI_CACHE_FIELDS])


def kvq_quantize_kivi(cfg: KiviConfig, axis: int, x, codes, scale, zero, tok_begin=0, stream=None):
    """x: fp16 [B][H][n_tok][D]."""
    _bits(x, (torch.float16,))
    B, H, n, D = x.shape
    c = cfg.to_c()
    _check(lib().kvq_quantize_kivi(ctypes.byref(c), axis, _ptr(x), H * n * D, n * D, B, n, _ptr(codes),
                                   _ptr(scale), _ptr(zero), tok_begin, _stream(stream)),
           "kvq_quantize_kivi")


def kvq_kivi_prefill(cfg: KiviConfig, cache: KiviCache, k, v, b0: int = 0, stream=None):
    """k, v: fp16 [B][H][n_tok][D] (same strides) for requests b0 .. b0+B-1."""
    _bits(k, (torch.float16,))
    _bits(v, (torch.float16,))
    if k.shape != v.shape or k.stride() != v.stride() or k.stride(3) != 1 or k.stride(2) != k.shape[3]:
        raise ValueError("k and v need one shape and rows of D contiguous channels")
    B, H, n, D = k.shape
    c = cfg.to_c()
    kc = cache.c_struct()
    _check(lib().kvq_kivi_prefill(ctypes.byref(c), ctypes.byref(kc), _ptr(k), _ptr(v), k.stride(0), k.stride(1),
                                  b0, B, n, _stream(stream)), "kvq_kivi_prefill")


def kvq_kivi_append(cfg: KiviConfig, cache: KiviCache, k_new, v_new, stream=None):
    """k_new, v_new: fp16 [n_seq][H][D], contiguous."""
    _bits(k_new, (torch.float16,))
    _bits(v_new, (torch.float16,))
    c = cfg.to_c()
    kc = cache.c_struct()
    _check(lib().kvq_kivi_append(ctypes.byref(c), ctypes.byref(kc), _ptr(k_new), _ptr(v_new), k_new.shape[0],
                                 _stream(stream)), "kvq_kivi_append")


class KiviCommitCall(_Call):
    """kvq_kivi_commit: k_draft, v_draft fp16 [n_seq][N][H][D], path int32 [n_seq][N], n_accept int32 [n_seq]."""

    def __init__(self, cfg: KiviConfig, cache: KiviCache, k_draft, v_draft, path, n_accept, stream=None):
        n_seq, N = path.shape
        for name, x in (("k_draft", k_draft), ("v_draft", v_draft)):
            _operand(name, x, (torch.float16,), (n_seq, N, cfg.n_heads, cfg.D))
        _operand("path", path, (torch.int32,), (n_seq, N))
        _operand("n_accept", n_accept, (torch.int32,), (n_seq,))
        c, kc = cfg.to_c(), cache.c_struct()
        super().__init__("kvq_kivi_commit", stream, path.device, (c, kc, cache, k_draft, v_draft, path, n_accept))
        self._bind(ctypes.byref(c), ctypes.byref(kc), _ptr(k_draft), _ptr(v_draft), _ptr(path), _ptr(n_accept),
                   n_seq, N)


def kvq_kivi_commit(cfg: KiviConfig, cache: KiviCache, k_draft, v_draft, path, n_accept, stream=None):
    """Append request b's drafted tokens path[b, :n_accept[b]] to the cache, in that order."""
    KiviCommitCall(cfg, cache, k_draft, v_draft, path, n_accept, stream)()


class KiviReadCall(_Call):
    """kvq_kivi_read into k_out and v_out (bf16, fp16 or fp32 [B][H][n_tok][D], rows of D contiguous channels
    packed along the tokens, one of them may be None); tok_begin int32 [B] or None."""

    def __init__(self, cfg: KiviConfig, cache: KiviCache, k_out, v_out, tok_begin=None, b0: int = 0, stream=None):
        x = k_out if k_out is not None else v_out
        if x is None:
            raise ValueError("neither k_out nor v_out is given")
        B, _, n, _ = x.shape
        for name, t in (("k_out", k_out), ("v_out", v_out)):
            if t is not None:
                _operand(name, t, tuple(_DT), (B, cfg.n_heads, n, cfg.D), contiguous=False)
                if t.stride(3) != 1 or (n > 1 and t.stride(2) != cfg.D):
                    raise ValueError(f"{name}: expected rows of D contiguous channels, packed along the tokens")
                if t.dtype != x.dtype or (_step(t, 0), _step(t, 1)) != (_step(x, 0), _step(x, 1)):
                    raise ValueError("k_out and v_out need one type and layout")
        if tok_begin is not None:
            _operand("tok_begin", tok_begin, (torch.int32,), (B,))
        c, kc = cfg.to_c(), cache.c_struct()
        super().__init__("kvq_kivi_read", stream, x.device, (c, kc, cache, k_out, v_out, tok_begin))
        self._bind(ctypes.byref(c), ctypes.byref(kc), _ptr(tok_begin), b0, B, n, _ptr(k_out), _ptr(v_out),
                   _DT[x.dtype], _step(x, 0), _step(x, 1))


def kvq_kivi_read(cfg: KiviConfig, cache: KiviCache, k_out, v_out, tok_begin=None, b0: int = 0, stream=None):
    """Read the cached tokens tok_begin[i] + j of requests b0 + i back into rows j of k_out and v_out."""
    KiviReadCall(cfg, cache, k_out, v_out, tok_begin, b0, stream)()


# ------------------------------------------------------------------------------------------
# Rows of queries, keys and values
# ------------------------------------------------------------------------------------------

def _rows(t: torch.Tensor | None):
    if t is None:
        return None
    return Rows(t.data_ptr(), _step(t, 0), _step(t, 1), _step(t, 2), t.shape[2], _DT[t.dtype])


class QkNormRopeCall(_Call):
    """kvq_qk_norm_rope over tensors [B][N][heads][D] of any strides with contiguous channels (views of a fused
    projection among them). q, k, v share a type; each may be None together with its output. w_q, w_k: [D] of that
    type. rope_cos, rope_sin: fp32 [max_ctx][D/2] or None; pos: int32 [B][N], None only without rotation."""

    def __init__(self, q, k, v, w_q, w_k, eps, rope_cos, rope_sin, pos, q_out, k_out, v_out, stream=None):
        x = next((t for t in (q, k, v) if t is not None), None)
        if x is None:
            raise ValueError("none of q, k and v is given")
        if x.dtype not in _DT:
            raise TypeError(f"expected one of {tuple(_DT)}, got {x.dtype}")
        B, N, _, D = x.shape
        for name, i, o in (("q", q, q_out), ("k", k, k_out), ("v", v, v_out)):
            if (i is None) != (o is None):
                raise ValueError(f"{name} needs both an input and an output")
            if i is not None:
                _operand(name, i, (x.dtype,), (B, N, None, D), contiguous=False)
                _operand(name + "_out", o, tuple(_DT), (B, N, i.shape[2], D), contiguous=False)
                if i.stride(3) != 1 or o.stride(3) != 1:
                    raise ValueError(f"{name}: the channels of a row need to be contiguous")
        for name, i, w in (("w_q", q, w_q), ("w_k", k, w_k)):
            if i is not None:
                if w is None:
                    raise ValueError(f"{name} is missing")
                _operand(name, w, (x.dtype,), (D,))
        if (rope_cos is None) != (rope_sin is None):
            raise ValueError("rope_cos and rope_sin go together")
        if rope_cos is not None:
            _operand("rope_cos", rope_cos, (torch.float32,), (None, D // 2))
            _operand("rope_sin", rope_sin, (torch.float32,), tuple(rope_cos.shape))
        if pos is not None:
            _operand("pos", pos, (torch.int32,), (B, N))
        rows = [_rows(t) for t in (q, k, v, q_out, k_out, v_out)]
        super().__init__("kvq_qk_norm_rope", stream, x.device,
                         (rows, q, k, v, w_q, w_k, rope_cos, rope_sin, pos, q_out, k_out, v_out))
        ref = [None if r is None else ctypes.byref(r) for r in rows]
        self._bind(D, B, N, *ref[:3], _ptr(w_q) if q is not None else None, _ptr(w_k) if k is not None else None,
                   float(eps), _ptr(rope_cos), _ptr(rope_sin), 0 if rope_cos is None else rope_cos.shape[0],
                   _ptr(pos), *ref[3:])


def kvq_qk_norm_rope(q, k, v, w_q, w_k, eps, rope_cos, rope_sin, pos, q_out, k_out, v_out, stream=None):
    """Norm of queries and keys for each head and the position rotation in one pass; values are converted."""
    QkNormRopeCall(q, k, v, w_q, w_k, eps, rope_cos, rope_sin, pos, q_out, k_out, v_out, stream)()


# ------------------------------------------------------------------------------------------
# Attention of drafted tokens
# ------------------------------------------------------------------------------------------

def kvq_kivi_tree_workspace_size(cfg: KiviConfig, B: int, N: int) -> int:
    c = cfg.to_c()
    return lib().kvq_kivi_tree_workspace_size(ctypes.byref(c), B, N)


def make_tree_workspace(cfg: KiviConfig, B: int, N: int, device="cuda") -> torch.Tensor:
    """A workspace for kvq_kivi_tree_attn (needs no initialisation; one for each call that runs at a time)."""
    return torch.empty(max(16, kvq_kivi_tree_workspace_size(cfg, B, N)), dtype=torch.uint8, device=device)


class _WorkspaceCall(_Call):
    """A call with a workspace, its last arguments but the stream. One that the caller does not give belongs to the
    stream of the call, and is made anew when the call runs on another one."""

    def _bind_ws(self, ws, make, device, *args):
        self._own = None  # the stream that a workspace of the call's own was allocated on
        if ws is None:
            with _on(self._keep[0], device):
                ws = self._ws = make()
            self._own = _stream(self._keep[0])
            self._again = make
        else:  # its bytes are what it says: contiguous, on the device
            _operand("ws", ws, (ws.dtype,), tuple(ws.shape))
            self._ws = ws
        self._bind(*args, _ptr(ws), ws.numel() * ws.element_size())

    def __call__(self):
        if self._own is not None and self._stream is None:
            s = torch._C._cuda_getCurrentRawStream(self._device)
            if s != self._own:  # called on another stream than before: a workspace that belongs there
                self._own, self._ws = s, self._again()
                self._args[-2] = ctypes.c_void_p(_ptr(self._ws))
        super().__call__()


class TreeAttnCall(_WorkspaceCall):
    """kvq_kivi_tree_attn: q bf16 [B][N][Hq][D], k_draft and v_draft fp16 [B][N][H][D], mask int64 (or uint64)
    [B][N] (bit j: drafted token j is seen), out bf16 or fp32 [B][N][Hq][D], n_draft int32 [B] or None (all N)."""

    def __init__(self, cfg: KiviConfig, cache: KiviCache, q, k_draft, v_draft, mask, out, n_draft=None, ws=None,
                 stream=None):
        B, N = mask.shape
        _operand("q", q, (torch.bfloat16,), (B, N, cfg.q_heads, cfg.D))
        _operand("out", out, (torch.bfloat16, torch.float32), tuple(q.shape))
        for name, x in (("k_draft", k_draft), ("v_draft", v_draft)):
            _operand(name, x, (torch.float16,), (B, N, cfg.n_heads, cfg.D))
        _operand("mask", mask, (torch.int64, torch.uint64), (B, N))
        if n_draft is not None:
            _operand("n_draft", n_draft, (torch.int32,), (B,))
        c, kc = cfg.to_c(), cache.c_struct()
        super().__init__("kvq_kivi_tree_attn", stream, q.device, (c, kc, cache, q, k_draft, v_draft, mask, out, n_draft, ws))
        args = (ctypes.byref(c), ctypes.byref(kc), _ptr(q), _ptr(k_draft), _ptr(v_draft), _ptr(mask),
                _ptr(n_draft), B, N, _ptr(out), OUT_FP32 if out.dtype == torch.float32 else OUT_BF16)
        self._bind_ws(ws, lambda: make_tree_workspace(cfg, B, N, q.device), q.device, *args)


def kvq_kivi_tree_attn(cfg: KiviConfig, cache: KiviCache, q, k_draft, v_draft, mask, out, n_draft=None, ws=None,
                       stream=None):
    """Attention of a tree of drafted tokens over the cache and one another. Without a workspace one is allocated
    for this call (through PyTorch, on the stream it runs on)."""
    TreeAttnCall(cfg, cache, q, k_draft, v_draft, mask, out, n_draft, ws, stream)()


# ------------------------------------------------------------------------------------------
# Attention under a shared prefix
# ------------------------------------------------------------------------------------------

def kvq_kivi_prefix_workspace_size(cfg: KiviConfig, prefix_cfg: KiviConfig, B: int, N: int) -> int:
    c, pc = cfg.to_c(), prefix_cfg.to_c()
    return lib().kvq_kivi_prefix_workspace_size(ctypes.byref(c), ctypes.byref(pc), B, N)


def make_prefix_workspace(cfg: KiviConfig, prefix_cfg: KiviConfig, B: int, N: int, device="cuda") -> torch.Tensor:
    """A workspace for kvq_kivi_prefix_attn (needs no initialisation; one for each call that runs at a time)."""
    return torch.empty(max(16, kvq_kivi_prefix_workspace_size(cfg, prefix_cfg, B, N)), dtype=torch.uint8, device=device)


class PrefixAttnCall(_WorkspaceCall):
    """kvq_kivi_prefix_attn: q bf16 [B][N][Hq][D], out bf16 or fp32 of that shape; ``prefix`` a KiviCache whose slot
    ``slot`` holds the tokens that every request of ``cache`` continues. k_draft and v_draft fp16 [B][N][H][D] and mask
    int64 (or uint64) [B][N] as in TreeAttnCall, or all None: no drafted tokens. n_draft int32 [B] or None (all N)."""

    def __init__(self, cfg: KiviConfig, cache: KiviCache, prefix_cfg: KiviConfig, prefix: KiviCache, slot: int, q, out,
                 k_draft=None, v_draft=None, mask=None, n_draft=None, ws=None, stream=None):
        if q.dim() != 4:
            raise ValueError(f"q: expected the shape (B, N, Hq, D), got {tuple(q.shape)}")
        B, N = q.shape[:2]
        _operand("q", q, (torch.bfloat16,), (B, N, cfg.q_heads, cfg.D))
        _operand("out", out, (torch.bfloat16, torch.float32), tuple(q.shape))
        if (k_draft is None) != (mask is None) or (v_draft is None) != (mask is None):
            raise ValueError("k_draft, v_draft and mask go together")
        if mask is not None:
            for name, x in (("k_draft", k_draft), ("v_draft", v_draft)):
                _operand(name, x, (torch.float16,), (B, N, cfg.n_heads, cfg.D))
            _operand("mask", mask, (torch.int64, torch.uint64), (B, N))
        if n_draft is not None:
            _operand("n_draft", n_draft, (torch.int32,), (B,))
        c, kc, pc, pk = cfg.to_c(), cache.c_struct(), prefix_cfg.to_c(), prefix.c_struct()
        super().__init__("kvq_kivi_prefix_attn", stream, q.device,
                         (c, kc, pc, pk, cache, prefix, q, k_draft, v_draft, mask, out, n_draft, ws))
        self._bind_ws(ws, lambda: make_prefix_workspace(cfg, prefix_cfg, B, N, q.device), q.device, ctypes.byref(c),
                      ctypes.byref(kc), ctypes.byref(pc), ctypes.byref(pk), slot, _ptr(q), _ptr(k_draft), _ptr(v_draft),
                      _ptr(mask), _ptr(n_draft), B, N, _ptr(out), OUT_FP32 if out.dtype == torch.float32 else OUT_BF16)


def kvq_kivi_prefix_attn(cfg: KiviConfig, cache: KiviCache, prefix_cfg: KiviConfig, prefix: KiviCache, slot: int, q, out,
                         k_draft=None, v_draft=None, mask=None, n_draft=None, ws=None, stream=None):
    """Attention of requests that continue one cached prefix: over the prefix, their own caches and their drafts.
    Without a workspace one is allocated for this call (through PyTorch, on the stream it runs on)."""
    PrefixAttnCall(cfg, cache, prefix_cfg, prefix, slot, q, out, k_draft, v_draft, mask, n_draft, ws, stream)()


# ------------------------------------------------------------------------------------------
# Slots of a cache
# ------------------------------------------------------------------------------------------

class CacheForkCall(_Call):
    """kvq_cache_fork: slot b0 + i of ``cache`` (VqCache or KiviCache) becomes what slot source[i] (int32 [n]) of
    ``from_cache`` was, or of ``cache`` itself without one; SLOT_KEEP and SLOT_FREE leave and empty a slot."""

    def __init__(self, cfg, cache, source, from_cfg=None, from_cache=None, b0: int = 0, stream=None):
        fmt, c = _fmt_cfg(cfg)
        if (from_cfg is None) != (from_cache is None):
            raise ValueError("from_cfg and from_cache go together")
        if from_cfg is not None and type(from_cfg) is not type(cfg):
            raise TypeError("caches of two formats")
        _operand("source", source, (torch.int32,), (None,))
        fc = None if from_cfg is None else _fmt_cfg(from_cfg)[1]
        kc, fk = cache.c_struct(), None if from_cache is None else from_cache.c_struct()
        super().__init__("kvq_cache_fork", stream, source.device, (c, kc, fc, fk, cache, from_cache, source))
        self._bind(fmt, ctypes.byref(c), ctypes.byref(kc), None if fc is None else ctypes.byref(fc),
                   None if fk is None else ctypes.byref(fk), _ptr(source), b0, source.shape[0])


def kvq_cache_fork(cfg, cache, source, from_cfg=None, from_cache=None, b0: int = 0, stream=None):
    """Slots of a cache continue other slots (fork, reorder, compact), or are freed."""
    CacheForkCall(cfg, cache, source, from_cfg, from_cache, b0, stream)()


# ------------------------------------------------------------------------------------------
# Verification of drafted tokens
# ------------------------------------------------------------------------------------------

def _dist(t: torch.Tensor | None):
    return None if t is None else Dist(t.data_ptr(), _step(t, 0), _step(t, 1), _DT[t.dtype])


class VerifyDraftCall(_Call):
    """kvq_verify_draft: target [B][N][V] (fp32, bf16 or fp16; any strides with contiguous entries), the target's
    probabilities behind every node, draft of that type and shape or None (point masses), token and parent int32 [B][N],
    u fp32 [B][N] or None (no sampling); path int32 [B][N], n_accept and next_token int32 [B] are written. n_draft int32
    [B] or None (all N)."""

    def __init__(self, target, draft, token, parent, u, path, n_accept, next_token, n_draft=None, stream=None):
        if target.dtype not in _DT:
            raise TypeError(f"target: expected one of {tuple(_DT)}, got {target.dtype}")
        if target.dim() != 3:
            raise ValueError(f"target: expected the shape (B, N, V), got {tuple(target.shape)}")
        B, N, V = target.shape
        for name, x in (("target", target), ("draft", draft)):
            if x is not None:
                _operand(name, x, (target.dtype,), (B, N, V), contiguous=False)
                if x.shape[2] > 1 and x.stride(2) != 1:
                    raise ValueError(f"{name}: the entries of a row need to be contiguous")
        for name, x in (("token", token), ("parent", parent), ("path", path)):
            _operand(name, x, (torch.int32,), (B, N))
        for name, x in (("n_accept", n_accept), ("next_token", next_token), ("n_draft", n_draft)):
            if x is not None or name != "n_draft":
                _operand(name, x, (torch.int32,), (B,))
        if u is not None:
            _operand("u", u, (torch.float32,), (B, N))
        p, q = _dist(target), _dist(draft)
        super().__init__("kvq_verify_draft", stream, target.device,
                         (p, q, target, draft, token, parent, u, path, n_accept, next_token, n_draft))
        self._bind(B, N, V, ctypes.byref(p), None if q is None else ctypes.byref(q), _ptr(token), _ptr(parent),
                   _ptr(n_draft), _ptr(u), _ptr(path), _ptr(n_accept), _ptr(next_token))


def kvq_verify_draft(target, draft, token, parent, u, path, n_accept, next_token, n_draft=None, stream=None):
    """Walk each request's tree of drafted tokens along the accepted ones and draw the token behind them."""
    VerifyDraftCall(target, draft, token, parent, u, path, n_accept, next_token, n_draft, stream)()


# ------------------------------------------------------------------------------------------
# Decode attention
# ------------------------------------------------------------------------------------------

def _fmt_cfg(cfg):
    if isinstance(cfg, VqConfig):
        return FMT_LOOPVQ, cfg.to_c()
    if isinstance(cfg, KiviConfig):
        return FMT_KIVI, cfg.to_c()
    raise TypeError(type(cfg))


def kvq_decode_workspace_size(cfg, B: int, n_splits: int = 0) -> int:
    fmt, c = _fmt_cfg(cfg)
    return lib().kvq_decode_workspace_size(fmt, ctypes.byref(c), B, n_splits)


def kvq_decode_auto_splits(cfg, B: int) -> int:
    fmt, c = _fmt_cfg(cfg)
    return lib().kvq_decode_auto_splits(fmt, ctypes.byref(c), B)


def make_workspace(cfg, B: int, n_splits: int = 0, device="cuda") -> torch.Tensor | None:
    n = kvq_decode_workspace_size(cfg, B, n_splits)
    if n == 0:
        return None
    return torch.zeros(n, dtype=torch.uint8, device=device)


class DecodeCall:
    """Pre-marshalled arguments of one repeated kvq_decode_attn call (cheap to launch)."""

    def __init__(self, cfg, cache, layer, loop_step, q, out, n_splits=0, ws=None, stream=None):
        self.fmt, self.cfg_c = _fmt_cfg(cfg)
        self.cache_c = cache.c_struct()
        _bits(q, (torch.bfloat16,))
        _bits(out, (torch.bfloat16, torch.float32))
        self.args = (self.fmt, ctypes.byref(self.cfg_c), ctypes.byref(self.cache_c), layer, loop_step,
                     _ptr(q), q.shape[0], _ptr(out), OUT_FP32 if out.dtype == torch.float32 else OUT_BF16,
                     n_splits, _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream))
        self._f = lib().kvq_decode_attn

    def __call__(self):
        st = self._f(*self.args)
        if st != KVQ_OK:
            _check(st, "kvq_decode_attn")


def kvq_decode_attn(cfg, cache, layer: int, loop_step: int, q, out, n_splits: int = 0, ws=None,
                    stream=None):
    """q: bf16 [B][H][D]; out: bf16 or fp32 [B][H][D]. When the split plan needs a workspace
    and none is given, a zero-filled one is allocated for this call (through PyTorch, on the
    stream it runs on)."""
    if ws is None:
        with _on(stream, q.device):
            ws = make_workspace(cfg, q.shape[0], n_splits, q.device)
    DecodeCall(cfg, cache, layer, loop_step, q, out, n_splits, ws, stream)()

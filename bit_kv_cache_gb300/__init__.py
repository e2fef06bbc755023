"""Python binding of libkvq (GB300 low-bit KV cache).

Argument marshalling only: every step of quantization, packing, buffer updates
and attention runs in the library's CUDA kernels, reached through the C ABI in
``include/kvq.h``.  PyTorch provides device memory and the current stream.  There
is no CPU fallback: importing this package fails if ``libkvq.so`` is missing
(build it with ``python bit_kv_cache_gb300/build.py``).
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libkvq.so")

KVQ_MODE_KIVI, KVQ_MODE_KITTY, KVQ_MODE_NVFP4, KVQ_MODE_E4M3, KVQ_MODE_INT8 = 0, 1, 2, 3, 4
KVQ_DEV_TIMEOUT, KVQ_DEV_BAD_STATE = 1, 2  # device status-word bits
STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported configuration",
          -3: "capacity exceeded", -4: "workspace missing or too small", -5: "CUDA error",
          -6: "device-side error reported"}
BUFFERS = ("k_codes", "k_hi", "k_bidx", "k_meta", "v_codes", "v_meta", "k_sink", "k_res",
           "v_res", "v_local")
EXPORTS = ("kvq_status_str", "kvq_config_check", "kvq_buffer_bytes", "kvq_quant_pack_k",
           "kvq_quant_pack_v", "kvq_append_token", "kvq_flush_group",
           "kvq_decode_attn_workspace_bytes", "kvq_workspace_init", "kvq_decode_attn",
           "kvq_read_status", "kvq_decode_attn_noalloc", "kvq_step_io_bytes", "kvq_decode_step_host",
           "kvq_decode_step_host_wait", "kvq_selftest_wait_timeout", "kvq_selftest_roles_timeout", "kvq_append_decode",
           "kvq_paged_bytes", "kvq_paged_init",
           "kvq_paged_prefill", "kvq_paged_append", "kvq_paged_flush_plan", "kvq_paged_flush",
           "kvq_paged_release", "kvq_paged_workspace_bytes", "kvq_paged_decode_attn",
           "kvq_paged_read_status", "kvq_paged_plan", "kvq_paged_chunk_workspace_bytes",
           "kvq_paged_chunk_attn", "kvq_paged_extend", "kvq_qk_norm_rope", "kvq_qk_norm_rope_freq",
           "kvq_paged_append_rope")
PAGED_MAX_B = 512


class KvqError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__("%s: %s (%d)" % (what, STATUS.get(code, "unknown"), code))
        self.code = code


class Config(ctypes.Structure):
    """kvq_config"""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "H_q", "H_kv", "D", "G", "bits", "S", "R",
                                              "n_boost", "mode", "v_bits")] + [("max_T", ctypes.c_int64)] + \
               [("rope", ctypes.c_int32), ("rope_base", ctypes.c_float)]


class Cache(ctypes.Structure):
    """kvq_cache"""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "k_hi", "k_bidx", "k_meta", "v_codes",
                                               "v_meta", "k_sink", "v_sink", "k_res", "v_res",
                                               "v_local", "status")] + \
               [(n, ctypes.c_int64) for n in ("n_sink", "T_k", "n_kres", "T_v", "n_vres",
                                              "n_local", "local_head")]


class Paged(ctypes.Structure):
    """kvq_paged"""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "k_meta", "v_codes", "v_meta")] + \
               [("n_pages", ctypes.c_int64)] + \
               [(n, ctypes.c_void_p) for n in ("page_table", "k_sink", "v_sink", "k_res", "v_res", "lens",
                                               "lens_host", "status")]


class ChunkDesc(ctypes.Structure):
    """kvq_chunk"""
    _fields_ = [(n, ctypes.c_void_p) for n in ("cu", "slot", "pos", "desc", "host")] + \
               [(n, ctypes.c_int64) for n in ("max_tokens", "n_tokens")] + [("captured", ctypes.c_int32)]


class QkConfig(ctypes.Structure):
    """kvq_qk_config"""
    _fields_ = [(n, ctypes.c_int32) for n in ("H_q", "H_kv", "D", "rotary_dim", "halves", "rotate")] + \
               [(n, ctypes.c_float) for n in ("eps", "rope_base")] + \
               [(n, ctypes.c_int64) for n in ("q_stride", "k_stride")]


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError("libkvq.so not built (%s); run: python bit_kv_cache_gb300/build.py" % path)
    L = ctypes.CDLL(path)
    P, I, I64, Sz, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    CP, KP, PP = ctypes.POINTER(Config), ctypes.POINTER(Cache), ctypes.POINTER(Paged)
    IP, HP = ctypes.POINTER(I), ctypes.POINTER(ChunkDesc)
    sig = {
        "kvq_status_str": ([I], ctypes.c_char_p),
        "kvq_config_check": ([CP], I),
        "kvq_buffer_bytes": ([CP, I], Sz),
        "kvq_quant_pack_k": ([CP, KP, P, I64, P], I),
        "kvq_quant_pack_v": ([CP, KP, P, I64, P], I),
        "kvq_append_token": ([CP, KP, P, P, P], I),
        "kvq_flush_group": ([CP, KP, ctypes.POINTER(I), ctypes.POINTER(I), P], I),
        "kvq_decode_attn_workspace_bytes": ([CP], Sz),
        "kvq_workspace_init": ([P, Sz, P], I),
        "kvq_decode_attn": ([CP, KP, P, P, P, Sz, P], I),
        "kvq_read_status": ([KP, P, ctypes.POINTER(ctypes.c_int32), P], I),
        "kvq_decode_attn_noalloc": ([CP, KP, P, P, P], I),
        "kvq_step_io_bytes": ([CP], Sz),
        "kvq_append_decode": ([CP, KP, P, P, P, P, P, Sz, IP, P], I),
        "kvq_decode_step_host": ([CP, KP, P, P, P, P, P, Sz, P, Sz, IP, IP, P], I),
        "kvq_decode_step_host_wait": ([CP, KP, P, P, P, P, P, P, Sz, IP, IP, P], I),
        "kvq_selftest_wait_timeout": ([P, P], I),
        "kvq_selftest_roles_timeout": ([P, P, P], I),
        "kvq_paged_bytes": ([CP, I64, I], Sz),
        "kvq_paged_init": ([CP, PP, P], I),
        "kvq_paged_prefill": ([CP, PP, I, P, P, I64, P], I),
        "kvq_paged_append": ([CP, PP, P, P, P], I),
        "kvq_paged_flush_plan": ([CP, PP, ctypes.POINTER(ctypes.c_int32), IP], I),
        "kvq_paged_flush": ([CP, PP, IP, P], I),
        "kvq_paged_release": ([CP, PP, I, P], I),
        "kvq_paged_workspace_bytes": ([CP], Sz),
        "kvq_paged_decode_attn": ([CP, PP, P, P, P, Sz, P], I),
        "kvq_paged_read_status": ([PP, P, ctypes.POINTER(ctypes.c_int32), P], I),
        "kvq_paged_plan": ([CP, PP, P, P, I64, HP, P], I),
        "kvq_paged_chunk_workspace_bytes": ([CP], Sz),
        "kvq_paged_chunk_attn": ([CP, PP, HP, P, I64, P, I64, P, I64, P, P, Sz, P], I),
        "kvq_paged_extend": ([CP, PP, HP, P, I64, P, I64, P], I),
        "kvq_qk_norm_rope": ([ctypes.POINTER(QkConfig), P, P, P, P, P, I64, P, P, P], I),
        "kvq_qk_norm_rope_freq": ([ctypes.POINTER(QkConfig), P, F, P, P, P, P, P, I64, P, P, P], I),
        "kvq_paged_append_rope": ([CP, PP, ctypes.POINTER(QkConfig), P, F, P, P, P, I64, P, P, P, P, I64, P], I),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    return L


lib = load_library()


def _check(code: int, what: str):
    if code != 0:
        raise KvqError(code, what)


def v_tile_tokens(cfg) -> int:
    """Tokens per value tile of a page (the library's value pages are tile-major): 256 /
    key bits when that divides G, else G."""
    t = 256 // (2 if cfg.mode == KVQ_MODE_KITTY else cfg.bits)
    return t if cfg.G % t == 0 else cfg.G


def make_config(B, H_q, H_kv, D, G, bits, S=0, R=None, n_boost=0, mode="kivi", max_T=0,
                v_bits=0, rope_base=0.0) -> Config:
    """rope_base > 0: keys are stored before RoPE and rotated in decode attention."""
    m = {"kivi": KVQ_MODE_KIVI, "kitty": KVQ_MODE_KITTY, "nvfp4": KVQ_MODE_NVFP4, "e4m3": KVQ_MODE_E4M3,
         "int8": KVQ_MODE_INT8}[mode]
    return Config(B, H_q, H_kv, D, G, bits, S, G if R is None else R, n_boost, m, v_bits or 0, max_T,
                  1 if rope_base else 0, float(rope_base or 0.0))


def _stream_of(index):
    """The current stream (cudaStream_t) of a device, which must be the current device."""
    import torch
    if torch._C._cuda_getDevice() != index:
        raise ValueError("the tensors are on cuda:%d, which is not the current device" % index)
    return torch._C._cuda_getCurrentRawStream(index)


def _index(device):
    """A device as Tensor.get_device() names it."""
    return -1 if device.index is None else device.index


def _rows(t, heads, D, n, device, what):
    """(address, row stride) of token-major rows [>= n][heads][D], float16, heads adjacent."""
    if t.get_device() != _index(device) or t.dtype is not _float16():
        raise ValueError("%s must be a float16 tensor on %s" % (what, device))
    if t.dim() != 3:
        raise ValueError("%s has shape %s, expected at least [%d, %d, %d]" % (what, tuple(t.shape), n, heads, D))
    (r, h, d), (s0, s1, s2) = t.shape, t.stride()
    if r < n or h != heads or d != D:
        raise ValueError("%s has shape %s, expected at least [%d, %d, %d]" % (what, (r, h, d), n, heads, D))
    if s2 != 1 or (heads > 1 and s1 != D):
        raise ValueError("%s must hold each token's heads contiguously" % what)
    return t.data_ptr(), (s0 if r > 1 else heads * D)


def _weight(w, D, device, what):
    """Address of a norm's weights (None: no norm)."""
    if w is None:
        return None
    if w.get_device() != _index(device) or w.dtype is not _float16() or w.dim() != 1 or w.numel() != D or not w.is_contiguous():
        raise ValueError("%s must be a contiguous float16 tensor [%d] on %s" % (what, D, device))
    return w.data_ptr()


_types = []


def _float16():
    if not _types:
        import torch
        _types.append(torch.float16)
    return _types[0]


class Rope:
    """Angles of a rotary position embedding: channel pair j of the first ``rotary_dim`` channels
    turns by pos * freq[j], and rotated channels are multiplied by ``amp``.  halves: pairs
    (j, j + rotary_dim/2) instead of (2j, 2j+1).  scaling: how positions beyond a model's
    training length are brought back into its range,
      None                                    freq[j] = base^(-2j/rotary_dim)
      dict(kind="linear", factor)             every frequency divided by factor
      dict(kind="ntk", factor)                a base larger by factor^(n/(n-2)): the last pair turns
                                              `factor` times slower, the first as before
      dict(kind="bands", factor, original, low=1.0, high=4.0)
                                              pairs that turn more than `high` times within
                                              `original` positions stay, those below `low` are
                                              divided by factor, in between linear in the turns
      dict(kind="yarn", factor, original, fast=32.0, slow=1.0)
                                              the same by a ramp over the pairs' indices, from the
                                              pair that turns `fast` times to the one of `slow`;
                                              amp = 0.1 ln(factor) + 1
    or ``freq`` gives the frequencies themselves (radians per position), with ``amp``."""

    def __init__(self, rotary_dim, base=10000.0, halves=False, scaling=None, freq=None, amp=None):
        n = int(rotary_dim)
        if n <= 0 or n % 2:
            raise ValueError("rotary_dim must be a positive even number")
        if freq is not None and scaling is not None:
            raise ValueError("freq and scaling exclude each other")
        gain = 1.0
        if freq is None:
            if not (math.isfinite(base) and base > 0):
                raise ValueError("base must be positive")
            freq, gain = self._frequencies(n, float(base), dict(scaling or {}))
        freq = [float(x) for x in freq]
        self.amp = float(gain if amp is None else amp)
        if len(freq) != n // 2 or not all(0 <= x <= 2.0 ** 31 for x in freq) or not math.isfinite(self.amp):
            raise ValueError("freq must hold rotary_dim / 2 frequencies of 0 to 2^31 radians, amp must be finite")
        self.rotary_dim, self.halves, self.freq = n, bool(halves), freq
        self._table = (ctypes.c_double * (n // 2))(*freq)
        self._ptr = ctypes.addressof(self._table)

    @staticmethod
    def _frequencies(n, base, scaling):
        kind = scaling.pop("kind", None)
        if kind is None and not scaling:
            return [base ** (-2.0 * j / n) for j in range(n // 2)], 1.0
        need = {"linear": {"factor"}, "ntk": {"factor"}, "bands": {"factor", "original"}, "yarn": {"factor", "original"}}
        may = {"bands": {"low": 1.0, "high": 4.0}, "yarn": {"fast": 32.0, "slow": 1.0}}
        if kind not in need or not need[kind] <= set(scaling) <= need[kind] | set(may.get(kind, ())):
            raise ValueError("unknown scaling: kind %r with %s" % (kind, sorted(scaling)))
        s = {m: float(x) for m, x in {**may.get(kind, {}), **scaling}.items()}
        if not all(math.isfinite(x) and x > 0 for x in s.values()):
            raise ValueError("the numbers of a scaling must be positive")
        k = s["factor"]
        if kind == "ntk":
            if n == 2:
                raise ValueError("one pair has no base to scale")
            base *= k ** (n / (n - 2))
        f = [base ** (-2.0 * j / n) for j in range(n // 2)]
        if kind == "ntk":
            return f, 1.0
        if kind == "linear":
            return [x / k for x in f], 1.0
        if kind == "bands":
            if s["high"] <= s["low"]:
                raise ValueError("high must be above low")
            keep = [(s["original"] * x / (2 * math.pi) - s["low"]) / (s["high"] - s["low"]) for x in f]
            gain = 1.0
        else:
            if base == 1.0:
                raise ValueError("a base of 1 has no pairs to choose from")
            at = lambda turns: n * math.log(s["original"] / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(math.floor(at(s["fast"])), 0), min(math.ceil(at(s["slow"])), n - 1)
            keep = [1 - (j - lo) / max(hi - lo, 0.001) for j in range(n // 2)]
            gain = 0.1 * math.log(k) + 1.0 if k > 1 else 1.0
        keep = [min(1.0, max(0.0, x)) for x in keep]
        return [x * p + x / k * (1 - p) for x, p in zip(f, keep)], gain


def qk_norm_rope(q, k=None, w_q=None, w_k=None, pos=None, eps=1e-6, rope_base=10000.0, rotary_dim=None,
                 halves=False, rotate_q=True, rotate_k=True, out=None, rope=None):
    """RMS norm of every query and key head and the rotary position embedding in one pass
    (kvq_qk_norm_rope).

    q: float16 [n, H_q, D]; k: float16 [n, H_kv, D] or None; rows may be strided (views of a
    fused projection).  w_q, w_k: float16 [D], or None for no norm.  pos: int32 [n] on the
    device.  rotary_dim: the first channels, which rotate (all of them by default); halves:
    pairs (j, j + rotary_dim/2) instead of (2j, 2j+1).  rotate_q, rotate_k: a cache that
    stores keys before RoPE takes rotate_k=False.  out: (q_out, k_out), contiguous; an
    output may be its own contiguous input.  rope: a Rope, instead of rope_base, rotary_dim and
    halves (kvq_qk_norm_rope_freq).  Returns (q_out, k_out)."""
    import torch
    n, H_q, D = q.shape
    dev = q.device
    H_kv = 0 if k is None else k.shape[1]
    qp, qs = _rows(q, H_q, D, n, dev, "q")
    kp, ks = (None, 0) if k is None else _rows(k, H_kv, D, n, dev, "k")
    if k is not None and k.shape[0] != n:
        raise ValueError("q and k have %d and %d rows" % (n, k.shape[0]))
    if pos is None or pos.device != dev or pos.dtype != torch.int32 or pos.shape != (n,) or not pos.is_contiguous():
        raise ValueError("pos must be a contiguous int32 tensor [%d] on %s" % (n, dev))
    for w, what in ((w_q, "w_q"), (w_k, "w_k")):
        if w is not None and (w.device != dev or w.dtype != torch.float16 or w.shape != (D,) or not w.is_contiguous()):
            raise ValueError("%s must be a contiguous float16 tensor [%d] on %s" % (what, D, dev))
    if out is None:
        out = (torch.empty((n, H_q, D), dtype=torch.float16, device=dev),
               None if k is None else torch.empty((n, H_kv, D), dtype=torch.float16, device=dev))
    q_out, k_out = out
    for y, H, what in ((q_out, H_q, "q_out"), (k_out, H_kv, "k_out")):
        if (y is None) != (what == "k_out" and k is None):
            raise ValueError("%s is %s" % (what, "missing" if y is None else "given without k"))
        if y is not None and (y.device != dev or y.dtype != torch.float16 or y.shape != (n, H, D) or not y.is_contiguous()):
            raise ValueError("%s must be a contiguous float16 tensor [%d, %d, %d] on %s" % (what, n, H, D, dev))
    c = QkConfig(H_q, H_kv, D, D if rotary_dim is None else rotary_dim, int(bool(halves)),
                 int(bool(rotate_q)) + 2 * int(bool(rotate_k)), eps, rope_base, qs, ks)
    if rope is not None:
        c.rotary_dim, c.halves = rope.rotary_dim, int(rope.halves)
        _check(lib.kvq_qk_norm_rope_freq(ctypes.byref(c), rope._ptr, rope.amp, qp, kp, None if w_q is None else w_q.data_ptr(),
                                         None if w_k is None else w_k.data_ptr(), pos.data_ptr(), n, q_out.data_ptr(),
                                         None if k_out is None else k_out.data_ptr(), _stream_of(dev.index)),
               "kvq_qk_norm_rope_freq")
        return q_out, k_out
    _check(lib.kvq_qk_norm_rope(ctypes.byref(c), qp, kp, None if w_q is None else w_q.data_ptr(),
                                None if w_k is None else w_k.data_ptr(), pos.data_ptr(), n, q_out.data_ptr(),
                                None if k_out is None else k_out.data_ptr(), _stream_of(dev.index)), "kvq_qk_norm_rope")
    return q_out, k_out


class KVQChunk:
    """The buffers of a plan (kvq_chunk) and of the attention that reads it: slot maps
    ``cu`` [B + 1], ``slot`` and ``pos`` [max_tokens] (int32, on the device).  Made by
    KVQPagedCache.new_chunk.  Every cache of the same configuration and lengths may attend
    with it; the cache that it was planned on last extends with it.  Two attention calls that
    may overlap, or captured ones whose replays may, need a chunk each.  A chunk whose
    attention was captured is not planned again: a replay reads its arrays."""

    def __init__(self, cfg, max_tokens, device):
        import torch
        i32 = dict(dtype=torch.int32, device=device)
        self.cu = torch.zeros(cfg.B + 1, **i32)
        self.slot = torch.zeros(max_tokens, **i32)
        self.pos = torch.zeros(max_tokens, **i32)
        self.desc = torch.zeros((cfg.B, 8), **i32)
        self.host = (ctypes.c_int32 * (8 * cfg.B))()
        self.ws = torch.empty(lib.kvq_paged_chunk_workspace_bytes(ctypes.byref(cfg)), dtype=torch.uint8, device=device)
        self.B, self.device = cfg.B, self.cu.device
        self.cache, self.mapping = None, 0  # the cache of the last plan, and its state of page mappings
        pad = torch.zeros(4, **i32) if max_tokens == 0 else None  # an empty tensor has no address
        self._pad = pad
        self.ws_ptr, self.ws_bytes = self.ws.data_ptr(), self.ws.numel()
        self.c = ChunkDesc(self.cu.data_ptr(), (self.slot if pad is None else pad).data_ptr(),
                           (self.pos if pad is None else pad).data_ptr(), self.desc.data_ptr(),
                           ctypes.cast(self.host, ctypes.c_void_p), max_tokens, 0, 0)
        self.ref = ctypes.byref(self.c)

    @property
    def n_tokens(self) -> int:
        return self.c.n_tokens


class KVQCache:
    """One attention layer's low-bit KV cache in device memory.

    Buffers are allocated with torch on ``device`` at the sizes the library reports
    (kvq_buffer_bytes); the library itself never allocates.  All calls enqueue on the
    current torch stream."""

    def __init__(self, B, H_q, H_kv, D, G, bits, S=0, R=None, n_boost=0, mode="kivi",
                 max_T=0, device="cuda", v_bits=0, rope_base=0.0):
        import torch
        self.torch = torch
        self.cfg = make_config(B, H_q, H_kv, D, G, bits, S, R, n_boost, mode, max_T, v_bits, rope_base)
        _check(lib.kvq_config_check(ctypes.byref(self.cfg)), "config")
        self.device = torch.device(device)
        self.c = Cache()
        self.buf = {}
        for i, name in enumerate(BUFFERS):
            n = lib.kvq_buffer_bytes(ctypes.byref(self.cfg), i)
            t = torch.zeros(max(n, 16), dtype=torch.uint8, device=self.device)
            self.buf[name] = t
            setattr(self.c, name, t.data_ptr() if n else None)
        self.device = t.device  # with its index, as the callers' tensors have it
        vs = torch.zeros(max(self.buf["k_sink"].numel(), 16), dtype=torch.uint8, device=self.device)
        self.buf["v_sink"] = vs
        self.c.v_sink = vs.data_ptr() if self.cfg.S else None
        self.status = torch.zeros(4, dtype=torch.int32, device=self.device)
        self.c.status = self.status.data_ptr()
        wsb = lib.kvq_decode_attn_workspace_bytes(ctypes.byref(self.cfg))
        self.ws = torch.zeros(wsb, dtype=torch.uint8, device=self.device)  # zero-filled
        # staging of kvq_decode_step_host (q, k_new, v_new, out of one step)
        self.io = torch.empty(lib.kvq_step_io_bytes(ctypes.byref(self.cfg)), dtype=torch.uint8,
                              device=self.device)
        self.done = None  # completion count of kvq_decode_step_host_wait (page-locked, made on first use)

    # -- helpers ------------------------------------------------------------- #
    @staticmethod
    def _stream():
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def _ptr(self, t, shape=None, what="tensor"):
        torch = self.torch
        if t.device != self.device or t.dtype != torch.float16 or not t.is_contiguous():
            raise ValueError("%s must be a contiguous float16 tensor on %s" % (what, self.device))
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError("%s has shape %s, expected %s" % (what, tuple(t.shape), tuple(shape)))
        return ctypes.c_void_p(t.data_ptr())

    @property
    def lengths(self) -> dict:
        c = self.c
        return dict(n_sink=c.n_sink, T_k=c.T_k, n_kres=c.n_kres, T_v=c.T_v, n_vres=c.n_vres,
                    n_local=c.n_local, local_head=c.local_head)

    @property
    def L(self) -> int:
        return self.c.n_sink + self.c.T_k + self.c.n_kres

    # -- the ABI ------------------------------------------------------------- #
    def quant_pack_k(self, k):
        B, Hkv, D = self.cfg.B, self.cfg.H_kv, self.cfg.D
        if k.dim() != 4 or tuple(k.shape[:2]) != (B, Hkv) or k.shape[3] != D:
            raise ValueError("k must be [B, H_kv, L0, D]")
        _check(lib.kvq_quant_pack_k(ctypes.byref(self.cfg), ctypes.byref(self.c),
                                    self._ptr(k, what="k"), k.shape[2], self._stream()),
               "kvq_quant_pack_k")

    def quant_pack_v(self, v):
        B, Hkv, D = self.cfg.B, self.cfg.H_kv, self.cfg.D
        if v.dim() != 4 or tuple(v.shape[:2]) != (B, Hkv) or v.shape[3] != D:
            raise ValueError("v must be [B, H_kv, L0, D]")
        _check(lib.kvq_quant_pack_v(ctypes.byref(self.cfg), ctypes.byref(self.c),
                                    self._ptr(v, what="v"), v.shape[2], self._stream()),
               "kvq_quant_pack_v")

    def prefill(self, k, v):
        self.quant_pack_k(k)
        self.quant_pack_v(v)

    def append_token(self, k_new, v_new):
        shp = (self.cfg.B, self.cfg.H_kv, self.cfg.D)
        _check(lib.kvq_append_token(ctypes.byref(self.cfg), ctypes.byref(self.c),
                                    self._ptr(k_new, shp, "k_new"), self._ptr(v_new, shp, "v_new"),
                                    self._stream()), "kvq_append_token")

    def flush_group(self) -> Tuple[bool, bool]:
        fk, fv = ctypes.c_int(0), ctypes.c_int(0)
        _check(lib.kvq_flush_group(ctypes.byref(self.cfg), ctypes.byref(self.c), ctypes.byref(fk),
                                   ctypes.byref(fv), self._stream()), "kvq_flush_group")
        return bool(fk.value), bool(fv.value)

    def decode_attn(self, q, out=None):
        torch = self.torch
        shp = (self.cfg.B, self.cfg.H_q, self.cfg.D)
        if out is None:
            out = torch.empty(shp, dtype=torch.float16, device=self.device)
        _check(lib.kvq_decode_attn(ctypes.byref(self.cfg), ctypes.byref(self.c),
                                   self._ptr(q, shp, "q"), self._ptr(out, shp, "out"),
                                   ctypes.c_void_p(self.ws.data_ptr()), self.ws.numel(),
                                   self._stream()), "kvq_decode_attn")
        return out

    def append_decode(self, q, k_new, v_new, out=None) -> Tuple[object, bool]:
        """Insert the token and attend (kvq_append_decode); returns (out, fused), fused
        telling whether one launch did both."""
        torch = self.torch
        shp, shk = (self.cfg.B, self.cfg.H_q, self.cfg.D), (self.cfg.B, self.cfg.H_kv, self.cfg.D)
        if out is None:
            out = torch.empty(shp, dtype=torch.float16, device=self.device)
        fused = ctypes.c_int(0)
        _check(lib.kvq_append_decode(ctypes.byref(self.cfg), ctypes.byref(self.c),
                                     self._ptr(k_new, shk, "k_new"), self._ptr(v_new, shk, "v_new"),
                                     self._ptr(q, shp, "q"), self._ptr(out, shp, "out"),
                                     ctypes.c_void_p(self.ws.data_ptr()), self.ws.numel(),
                                     ctypes.byref(fused), self._stream()), "kvq_append_decode")
        return out, bool(fused.value)

    def step(self, q, k_new, v_new, out=None):
        """One decode step in the Kitty pipeline order: insert, attend, flush."""
        out, _ = self.append_decode(q, k_new, v_new, out)
        self.flush_group()
        return out

    def step_host(self, q, k_new, v_new, out, wait=False):
        """One decode step from host tensors (kvq_decode_step_host): q, out [B, H_q, D],
        k_new, v_new [B, H_kv, D], contiguous float16 on the CPU (page-locked for the
        copies to be asynchronous).  Enqueued on the current stream; out holds the
        result once the stream is synchronized.  wait (kvq_decode_step_host_wait; all
        four tensors page-locked): returns once out holds the result.  Returns
        (flushed_k, flushed_v)."""
        torch = self.torch
        for t, shp, what in ((q, (self.cfg.B, self.cfg.H_q, self.cfg.D), "q"),
                             (out, (self.cfg.B, self.cfg.H_q, self.cfg.D), "out"),
                             (k_new, (self.cfg.B, self.cfg.H_kv, self.cfg.D), "k_new"),
                             (v_new, (self.cfg.B, self.cfg.H_kv, self.cfg.D), "v_new")):
            if t.device.type != "cpu" or t.dtype != torch.float16 or not t.is_contiguous() or \
                    tuple(t.shape) != shp:
                raise ValueError("%s must be a contiguous float16 CPU tensor of shape %s" % (what, shp))
        fk, fv = ctypes.c_int(0), ctypes.c_int(0)
        if wait:
            if self.done is None:
                self.done = torch.zeros(1, dtype=torch.int32).pin_memory()
            _check(lib.kvq_decode_step_host_wait(ctypes.byref(self.cfg), ctypes.byref(self.c),
                                                 ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k_new.data_ptr()),
                                                 ctypes.c_void_p(v_new.data_ptr()), ctypes.c_void_p(out.data_ptr()),
                                                 ctypes.c_void_p(self.done.data_ptr()),
                                                 ctypes.c_void_p(self.ws.data_ptr()), self.ws.numel(),
                                                 ctypes.byref(fk), ctypes.byref(fv), self._stream()),
                   "kvq_decode_step_host_wait")
            return bool(fk.value), bool(fv.value)
        _check(lib.kvq_decode_step_host(ctypes.byref(self.cfg), ctypes.byref(self.c),
                                        ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k_new.data_ptr()),
                                        ctypes.c_void_p(v_new.data_ptr()), ctypes.c_void_p(out.data_ptr()),
                                        ctypes.c_void_p(self.io.data_ptr()), self.io.numel(),
                                        ctypes.c_void_p(self.ws.data_ptr()), self.ws.numel(),
                                        ctypes.byref(fk), ctypes.byref(fv), self._stream()),
               "kvq_decode_step_host")
        return bool(fk.value), bool(fv.value)

    def read_status(self) -> int:
        st = ctypes.c_int32(0)
        lib.kvq_read_status(ctypes.byref(self.c), ctypes.c_void_p(self.ws.data_ptr()),
                            ctypes.byref(st), self._stream())
        return st.value

    # -- typed views of the buffers (for inspection and tests) ---------------- #
    def view(self, name: str):
        torch = self.torch
        cfg = self.cfg
        U, D, T, G = cfg.B * cfg.H_kv, cfg.D, cfg.max_T, cfg.G
        kitty = cfg.mode == KVQ_MODE_KITTY
        if cfg.mode == KVQ_MODE_NVFP4:  # codes [B][H][T][D/2]; page records of 16 + G*D/16 bytes
            b = self.buf[name]
            ms = 16 + G * D // 16
            if name in ("k_codes", "v_codes"):
                return b[: U * T * D // 2].view(cfg.B, cfg.H_kv, T, D // 2)
            if name in ("k_meta", "v_meta"):
                return b[: U * (T // G) * ms].view(cfg.B, cfg.H_kv, T // G, ms)
        kfpi = 16 if kitty else 32 // cfg.bits
        vfpi = 32 // (cfg.v_bits or cfg.bits)
        Gv = min(G, D)
        b = self.buf[name]
        if name == "k_codes":
            return b.view(torch.int32).view(cfg.B, cfg.H_kv, T // kfpi, D)
        if name == "k_hi":
            return b[: U * (T // 16) * cfg.n_boost * 4].view(torch.int32).view(cfg.B, cfg.H_kv, T // 16, cfg.n_boost)
        if name == "k_bidx":
            return b[: U * (T // G) * D].view(cfg.B, cfg.H_kv, T // G, D)
        if name == "k_meta":
            return b.view(torch.float16).view(cfg.B, cfg.H_kv, T // G, D, 2)
        if name == "v_codes":  # tile-major pages: [G / TV][D / fpi rows][TV words]
            TV = v_tile_tokens(cfg)
            return b.view(torch.int32).view(cfg.B, cfg.H_kv, T // G, G // TV, D // vfpi, TV)
        if name == "v_meta":
            return b.view(torch.float16).view(cfg.B, cfg.H_kv, T, D // Gv, 2)
        rows = {"k_sink": cfg.S, "v_sink": cfg.S, "k_res": G if kitty else cfg.R,
                "v_res": G if kitty else cfg.R, "v_local": cfg.R if kitty else 0}[name]
        return b[: U * rows * D * 2].view(torch.float16).view(cfg.B, cfg.H_kv, rows, D)


class KVQPagedCache:
    """A paged low-bit KV cache: B batch slots of their own lengths over a pool of n_pages
    physical pages, each holding one group of G tokens of all H_kv heads of one slot.  The
    page table and the pool live in torch device memory; this class keeps the free list on
    the host and writes the table rows a slot needs before the library packs into them
    (prefill, flush).  ``max_T`` is the packed-token capacity of one slot.  mode: "kivi"
    (min-max codes of 2, 4 or 8 bits), or "e4m3" and "int8" (bits=8): codes of that type with
    one scale for each page and head, on their own for keys and values."""

    def __init__(self, B, H_q, H_kv, D, G, bits, n_pages, max_T, S=0, R=None, device="cuda", v_bits=0, mode="kivi"):
        import torch
        self.torch = torch
        self.cfg = make_config(B, H_q, H_kv, D, G, bits, S, R, 0, mode, max_T, v_bits)
        self.device = torch.device(device)
        self.n_pages = n_pages
        cp = ctypes.byref(self.cfg)
        self.p = Paged()
        self.buf = {}
        for name, which in (("k_codes", 0), ("k_meta", 3), ("v_codes", 4), ("v_meta", 5), ("k_sink", 6),
                            ("v_sink", 6), ("k_res", 7), ("v_res", 8)):
            n = lib.kvq_paged_bytes(cp, n_pages, which)
            if n == 0 and which in (0, 3, 4, 5, 7, 8) and n_pages > 0:
                raise KvqError(-2, "paged config")
            t = torch.zeros(max(n, 16), dtype=torch.uint8, device=self.device)
            self.buf[name] = t
            setattr(self.p, name, t.data_ptr() if n else None)
        self.device = self._dev = t.device  # with its index, as the callers' tensors have it
        self.max_pages = max_T // G
        self.table = torch.zeros((B, self.max_pages), dtype=torch.int32, device=self.device)
        self.lens = torch.zeros((B, 4), dtype=torch.int32, device=self.device)
        self.lens_host = (ctypes.c_int32 * (4 * B))()
        self.status = torch.zeros(4, dtype=torch.int32, device=self.device)
        self.p.n_pages = n_pages
        self.p.page_table = self.table.data_ptr()
        self.p.lens = self.lens.data_ptr()
        self.p.lens_host = ctypes.cast(self.lens_host, ctypes.c_void_p)
        self.p.status = self.status.data_ptr()
        self.ws = torch.zeros(lib.kvq_paged_workspace_bytes(cp), dtype=torch.uint8, device=self.device)
        self._refs = ctypes.byref(self.cfg), ctypes.byref(self.p)
        self._ws = self.ws.data_ptr(), self.ws.numel()
        self._dims, self._rope = (B, H_q, H_kv, D), None
        self.caller_pages = False                     # plan() was given pages of the caller's
        self.mapping = 0                              # counts the calls that took pages away from slots
        self.free = list(range(n_pages - 1, -1, -1))  # pop() hands out the lowest id first
        self.pages = [[] for _ in range(B)]           # physical pages of each slot, logical order
        _check(lib.kvq_paged_init(cp, ctypes.byref(self.p), KVQCache._stream()), "paged init")

    def _ptr(self, t, shape, what):
        return KVQCache._ptr(self, t, shape, what)

    def lengths(self, b) -> dict:
        l = self.lens_host[4 * b: 4 * b + 4]
        return {"n_sink": l[0], "T": l[1], "n_res": l[2], "active": l[3]}

    def _map(self, b, n):
        """Maps the next n logical pages of slot b to free physical pages."""
        if n == 0:
            return
        if self.caller_pages:
            raise KvqError(-1, "the caller maps this cache's pages")
        if len(self.free) < n:
            raise KvqError(-3, "page pool exhausted")
        j0 = len(self.pages[b])
        new = [self.free.pop() for _ in range(n)]
        self.pages[b].extend(new)
        self.table[b, j0:j0 + n] = self.torch.tensor(new, dtype=self.torch.int32)

    def prefill(self, b, k, v):
        """k, v: float16 [H_kv][L0][D] of batch slot b (empty)."""
        cfg = self.cfg
        L0 = k.shape[1]
        self._ptr(k, (cfg.H_kv, L0, cfg.D), "k")
        self._ptr(v, (cfg.H_kv, L0, cfg.D), "v")
        if self.lens_host[4 * b + 3]:
            raise KvqError(-1, "prefill of an occupied slot")
        ns = min(cfg.S, L0)
        self._map(b, max(0, (L0 - ns) // cfg.G - len(self.pages[b])))
        _check(lib.kvq_paged_prefill(ctypes.byref(self.cfg), ctypes.byref(self.p), b, ctypes.c_void_p(k.data_ptr()),
                                     ctypes.c_void_p(v.data_ptr()), L0, KVQCache._stream()), "paged prefill")

    def append(self, k_new, v_new):
        cfg = self.cfg
        kp = self._ptr(k_new, (cfg.B, cfg.H_kv, cfg.D), "k_new")
        vp = self._ptr(v_new, (cfg.B, cfg.H_kv, cfg.D), "v_new")
        _check(lib.kvq_paged_append(ctypes.byref(self.cfg), ctypes.byref(self.p), kp, vp, KVQCache._stream()),
               "paged append")

    def append_rope(self, q, k, v, rope=None, w_q=None, w_k=None, eps=1e-6, rotate_q=True, rotate_k=True, pages=None,
                    out=None):
        """One new token for every active slot: full residuals are packed, the queries and keys
        are normalized (w_q, w_k: float16 [D], or None for no norm) and rotated at the tokens'
        positions, and keys and values enter the cache, in one launch (kvq_paged_append_rope).
        q: float16 [B, H_q, D], k, v: float16 [B, H_kv, D], row b for slot b; rows may be strided
        (views of a fused projection), those of empty slots are ignored.  rope: a Rope; by
        default all channels, interleaved, base 10000.  pages: ids of physical pages that the
        caller hands out to the full residuals (host integers, or an int32 CPU tensor; pages that
        no slot holds, each once), here and in every later call that needs pages, until clear(); by
        default they come from the
        cache's own free list.  Returns the queries for decode_attn, out if it is given
        (contiguous [B, H_q, D]; it may be q)."""
        dev = self._dev
        B, H_q, H_kv, D = self._dims
        qp, qs = _rows(q, H_q, D, B, dev, "q")
        kp, ks = _rows(k, H_kv, D, B, dev, "k")
        vp, vs = _rows(v, H_kv, D, B, dev, "v")
        wq, wk = _weight(w_q, D, dev, "w_q"), _weight(w_k, D, dev, "w_k")
        if out is None:
            if self.torch.cuda.is_current_stream_capturing():
                raise KvqError(-2, "kvq_paged_append_rope")  # before anything is allocated
            out = self.torch.zeros((B, H_q, D), dtype=self.torch.float16, device=dev)
        op, os_ = _rows(out, H_q, D, B, dev, "out")
        if os_ != H_q * D or out.numel() != B * H_q * D:
            raise ValueError("out must be contiguous [%d, %d, %d]" % (B, H_q, D))
        if rope is None:
            rope = self._rope = self._rope or Rope(D)
        c = QkConfig(H_q, H_kv, D, rope.rotary_dim, rope.halves, (1 if rotate_q else 0) + (2 if rotate_k else 0), eps, 0.0, qs, ks)
        own, taken = pages is None, ()
        if own:
            pp, np_, taken = self._full_pages()
        elif isinstance(pages, self.torch.Tensor):
            if pages.get_device() >= 0 or pages.dtype is not self.torch.int32 or pages.dim() != 1 or not pages.is_contiguous():
                raise ValueError("pages must be a contiguous int32 CPU tensor")
            pp, np_ = (pages.data_ptr() or ctypes.addressof(self.lens_host)), pages.numel()
        else:
            ids = (ctypes.c_int32 * max(1, len(pages)))(*[int(x) for x in pages])
            pp, np_ = ids, len(pages)
        try:
            _check(lib.kvq_paged_append_rope(*self._refs, ctypes.byref(c), rope._ptr, rope.amp, qp, kp, vp, vs, wq, wk, op, pp, np_,
                                             _stream_of(dev.index)), "kvq_paged_append_rope")
        except Exception:
            for b in reversed(taken):  # their table rows are not written
                self.free.append(self.pages[b].pop())
            raise
        self.caller_pages |= not own
        return out

    def _full_pages(self):
        """Pages for the full residuals, slot after slot, from the free list: (ids, their number,
        the slots that got one each time)."""
        cfg = self.cfg
        n, seqs = ctypes.c_int(0), (ctypes.c_int32 * cfg.B)()
        _check(lib.kvq_paged_flush_plan(*self._refs, seqs, ctypes.byref(n)), "flush plan")
        ids, taken, per, full = [], [], cfg.R // cfg.G, seqs[: n.value]
        if full and self.caller_pages:
            raise KvqError(-1, "the caller maps this cache's pages")
        j0 = [self.lens_host[4 * b + 1] // cfg.G for b in full]
        if sum(max(0, j + per - len(self.pages[b])) for b, j in zip(full, j0)) > len(self.free):
            raise KvqError(-3, "page pool exhausted")
        for b, j in zip(full, j0):
            while len(self.pages[b]) < j + per:
                taken.append(b)
                self.pages[b].append(self.free.pop())
            ids += self.pages[b][j: j + per]
        return (ctypes.c_int32 * len(ids))(*ids), len(ids), taken

    def decode_step(self, q, k, v, rope=None, w_q=None, w_k=None, eps=1e-6, out=None):
        """One decode step of every active slot: append_rope, then decode_attn."""
        return self.decode_attn(self.append_rope(q, k, v, rope, w_q, w_k, eps), out)

    def flush(self) -> list:
        """Packs every full residual into new pages; returns the flushed slots."""
        cfg = self.cfg
        seqs = (ctypes.c_int32 * cfg.B)()
        n = ctypes.c_int(0)
        _check(lib.kvq_paged_flush_plan(ctypes.byref(self.cfg), ctypes.byref(self.p), seqs, ctypes.byref(n)),
               "flush plan")
        out = list(seqs[: n.value])
        for b in out:
            self._map(b, max(0, (self.lens_host[4 * b + 1] + cfg.R) // cfg.G - len(self.pages[b])))
        nf = ctypes.c_int(0)
        _check(lib.kvq_paged_flush(ctypes.byref(self.cfg), ctypes.byref(self.p), ctypes.byref(nf),
                                   KVQCache._stream()), "paged flush")
        return out

    def release(self, b):
        self.mapping += len(self.pages[b]) > 0
        self.free.extend(reversed(self.pages[b]))
        self.pages[b] = []
        _check(lib.kvq_paged_release(ctypes.byref(self.cfg), ctypes.byref(self.p), b, KVQCache._stream()),
               "paged release")

    def clear(self, unmap=True):
        """Empties every slot and unmaps its pages; the cache maps its own again if the caller
        did.  unmap=False: the pages stay mapped to their slots, which refill them."""
        _check(lib.kvq_paged_init(*self._refs, _stream_of(self._dev.index)),
               "paged init")
        if unmap:
            self.mapping += 1
            self.caller_pages = False
            for b in range(self.cfg.B - 1, -1, -1):
                self.free.extend(reversed(self.pages[b]))
                self.pages[b] = []

    # -- chunks of new tokens ------------------------------------------------- #
    def new_chunk(self, max_tokens) -> KVQChunk:
        """Buffers for plans of up to max_tokens new tokens."""
        return KVQChunk(self.cfg, max_tokens, self._dev)

    def _check_chunk(self, chunk):
        """The library reads a row of the chunk's arrays for each of this cache's slots."""
        if chunk.B != self.cfg.B or chunk.device != self._dev:
            raise ValueError("the chunk belongs to another configuration")

    def plan(self, n_new, chunk=None, pages=None) -> KVQChunk:
        """Plans n_new[b] new tokens for every slot (kvq_paged_plan): slot maps, positions,
        and the page-table rows of the pages that extend() will pack.  n_new: B integers, or
        an int32 CPU tensor.  pages: int32 device tensor of physical pages that the caller
        hands out, in the order slots need them, here and in every later call that needs pages,
        until clear(); by default they come from the cache's own free list."""
        torch, cfg = self.torch, self.cfg
        if isinstance(n_new, torch.Tensor):
            if n_new.device.type != "cpu" or n_new.dtype != torch.int32 or n_new.shape != (cfg.B,) or not n_new.is_contiguous():
                raise ValueError("n_new must be a contiguous int32 CPU tensor [%d]" % cfg.B)
            np_ = n_new.data_ptr()
        else:
            n_new = [int(x) for x in n_new]
            if len(n_new) != cfg.B or any(not 0 <= x < 1 << 31 for x in n_new):
                raise ValueError("n_new must hold %d counts" % cfg.B)
            np_ = (ctypes.c_int32 * cfg.B)(*n_new)
        if chunk is not None:
            self._check_chunk(chunk)
        if (chunk is None or pages is None) and torch.cuda.is_current_stream_capturing():
            raise KvqError(-2, "kvq_paged_plan")  # before anything is allocated or copied
        if chunk is None:
            chunk = self.new_chunk(int(sum(n_new)))
        taken = []  # (slot, page) handed out here
        planned = pages is None
        if not planned and (pages.device != self._dev or pages.dtype != torch.int32 or pages.dim() != 1 or
                            not pages.is_contiguous()):
            raise ValueError("pages must be a contiguous int32 tensor on %s" % self._dev)
        try:
            if planned:
                pages = self._plan_pages(n_new.tolist() if isinstance(n_new, torch.Tensor) else n_new, taken)
            _check(lib.kvq_paged_plan(*self._refs, np_, None if pages is None else pages.data_ptr(),
                                      0 if pages is None else pages.numel(), chunk.ref, _stream_of(self._dev.index)),
                   "kvq_paged_plan")
        except Exception:
            for b, page in reversed(taken):  # their table rows are not written
                self.pages[b].pop()
                self.free.append(page)
            raise
        self.caller_pages |= not planned
        chunk.cache, chunk.mapping = self, self.mapping
        return chunk

    def _plan_pages(self, n_new, taken):
        """Physical pages of a plan, from the free list: logical pages [T/G, ...) of each
        slot that packs, as a device tensor (None: no slot packs); those that the slot did not
        have are appended to taken."""
        cfg = self.cfg
        todo = []
        for b, n in enumerate(n_new):
            ns, T, nr, on = self.lens_host[4 * b: 4 * b + 4]
            if n <= 0:
                continue
            if not on:
                ns = T = nr = 0
            pk = (nr + n - min(n, cfg.S - ns)) // cfg.R * cfg.R
            if pk and T + pk <= cfg.max_T:  # a longer one is refused by the library
                todo.append((b, T // cfg.G, (T + pk) // cfg.G))
        if not todo:
            return None
        if self.caller_pages:
            raise KvqError(-1, "the caller maps this cache's pages")
        if sum(max(0, hi - len(self.pages[b])) for b, lo, hi in todo) > len(self.free):
            raise KvqError(-3, "page pool exhausted")
        ids = []
        for b, lo, hi in todo:
            while len(self.pages[b]) < hi:
                taken.append((b, self.free.pop()))
                self.pages[b].append(taken[-1][1])
            ids += self.pages[b][lo:hi]
        t = self.torch.tensor(ids, dtype=self.torch.int32).pin_memory()
        return t.to(self._dev, non_blocking=True)

    def chunk_attn(self, chunk, q, k_new, v_new, out=None):
        """Attention of the planned chunk's tokens over the cached tokens and, causally, the
        chunk (kvq_paged_chunk_attn).  q: float16 [n, H_q, D], k_new, v_new: float16
        [n, H_kv, D], n >= chunk.n_tokens, token-major rows that may be strided; rows behind
        chunk.n_tokens are left alone.  The cache is not changed."""
        self._check_chunk(chunk)
        torch, cfg, dev, n = self.torch, self.cfg, self._dev, chunk.n_tokens
        qp, qs = _rows(q, cfg.H_q, cfg.D, n, dev, "q")
        kp, ks = _rows(k_new, cfg.H_kv, cfg.D, n, dev, "k_new")
        vp, vs = _rows(v_new, cfg.H_kv, cfg.D, n, dev, "v_new")
        if out is None:
            out = (torch.empty if q.shape[0] == n else torch.zeros)(q.shape, dtype=torch.float16, device=dev)
        op, os_ = _rows(out, cfg.H_q, cfg.D, n, dev, "out")
        if os_ != cfg.H_q * cfg.D:
            raise ValueError("out must be contiguous")
        _check(lib.kvq_paged_chunk_attn(*self._refs, chunk.ref, qp, qs, kp, ks, vp, vs, op, chunk.ws_ptr, chunk.ws_bytes,
                                        _stream_of(dev.index)), "kvq_paged_chunk_attn")
        return out

    def extend(self, chunk, k_new, v_new):
        """The planned chunk's tokens enter the cache (kvq_paged_extend).  The chunk must have
        been planned on this cache, which maps the pages, unless the caller maps them."""
        cfg, dev = self.cfg, self._dev
        self._check_chunk(chunk)
        if chunk.cache is not self and not self.caller_pages:
            raise KvqError(-1, "the chunk was planned on another cache")
        if chunk.mapping != self.mapping and not self.caller_pages:
            raise KvqError(-1, "pages were released since the plan")
        kp, ks = _rows(k_new, cfg.H_kv, cfg.D, chunk.n_tokens, dev, "k_new")
        vp, vs = _rows(v_new, cfg.H_kv, cfg.D, chunk.n_tokens, dev, "v_new")
        _check(lib.kvq_paged_extend(*self._refs, chunk.ref, kp, ks, vp, vs, _stream_of(dev.index)), "kvq_paged_extend")

    def chunk_step(self, n_new, q, k, v, w_q=None, w_k=None, eps=1e-6, rope_base=10000.0, rotary_dim=None,
                   halves=False, chunk=None, out=None, rope=None):
        """One step of n_new[b] new tokens per slot: plan, norm and rotation of q and k at
        their positions, attention, and the tokens' entry into the cache.  q: float16
        [n, H_q, D], k, v: float16 [n, H_kv, D], n >= sum(n_new); rows behind that sum are left
        alone.  rope: a Rope, instead of rope_base, rotary_dim and halves.  Returns (out, chunk),
        out with sum(n_new) rows if it is not the caller's.  A chunk made here (chunk=None) costs
        its arrays and a workspace in every call; a loop keeps one."""
        chunk = self.plan(n_new, chunk)
        n = chunk.n_tokens
        if n == 0:
            return q.new_empty((0,) + q.shape[1:]) if out is None else out, chunk
        q, k = qk_norm_rope(q[:n], k[:n], w_q, w_k, chunk.pos[:n], eps, rope_base, rotary_dim, halves, rope=rope)
        out = self.chunk_attn(chunk, q, k, v, out)
        self.extend(chunk, k, v)
        return out, chunk

    def decode_attn(self, q, out=None):
        """Attention of one query token per active slot over its cached tokens
        (kvq_paged_decode_attn).  q, out: float16 [B, H_q, D], contiguous; rows of empty slots are
        not written (zeros where out is made here).  The cache's workspace serves one call at a
        time: calls on streams that may overlap, or replays of captured ones, must be ordered."""
        cfg, dev = self.cfg, self._dev
        shape = (cfg.B, cfg.H_q, cfg.D)
        if out is None:
            out = self.torch.zeros_like(q)
        for t, what in ((q, "q"), (out, "out")):
            if t.get_device() != _index(dev) or t.dtype is not _float16() or not t.is_contiguous():
                raise ValueError("%s must be a contiguous float16 tensor on %s" % (what, dev))
            if t.shape != shape:
                raise ValueError("%s has shape %s, expected %s" % (what, tuple(t.shape), shape))
        _check(lib.kvq_paged_decode_attn(*self._refs, q.data_ptr(), out.data_ptr(), *self._ws, _stream_of(dev.index)),
               "paged decode")
        return out

    def read_status(self) -> int:
        st = ctypes.c_int32(0)
        lib.kvq_paged_read_status(ctypes.byref(self.p), ctypes.c_void_p(self.ws.data_ptr()), ctypes.byref(st),
                                  KVQCache._stream())
        return st.value

    def view(self, name: str):
        """Typed views of the page pools ([n_pages][H_kv] ...) and the fp16 buffers."""
        torch = self.torch
        cfg = self.cfg
        P, H, D, G = self.n_pages, cfg.H_kv, cfg.D, cfg.G
        kfpi, vfpi, Gv = 32 // cfg.bits, 32 // (cfg.v_bits or cfg.bits), min(G, D)
        b = self.buf[name]
        if cfg.mode in (KVQ_MODE_E4M3, KVQ_MODE_INT8):
            code = torch.float8_e4m3fn if cfg.mode == KVQ_MODE_E4M3 else torch.int8
            if name == "k_codes":  # 16-byte chunk j of row t at position j ^ (4 * (t mod 2))
                return b[: P * H * G * D].view(code).view(P, H, G, D)
            if name == "v_codes":
                return b[: P * H * G * D].view(code).view(P, H, G // 64, D, 64)
            if name in ("k_meta", "v_meta"):  # the scales
                return b[: P * H * 16].view(torch.float32).view(P, H, 4)[..., 0]
        if name == "k_codes":
            return b.view(torch.int32).view(P, H, G // kfpi, D)
        if name == "k_meta":
            return b.view(torch.float16).view(P, H, D, 2)
        if name == "v_codes":  # tile-major pages: [G / TV][D / fpi rows][TV words]
            TV = v_tile_tokens(cfg)
            return b.view(torch.int32).view(P, H, G // TV, D // vfpi, TV)
        if name == "v_meta":
            return b.view(torch.float16).view(P, H, G, D // Gv, 2)
        rows = {"k_sink": cfg.S, "v_sink": cfg.S, "k_res": cfg.R, "v_res": cfg.R}[name]
        return b[: cfg.B * H * rows * D * 2].view(torch.float16).view(cfg.B, H, rows, D)

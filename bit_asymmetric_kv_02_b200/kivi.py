"""ctypes binding of the CUDA library ``libkivi.so`` (C ABI in include/kivi.h).

Argument marshalling only: every computation runs in the library's kernels.  Functions keep the C
names.  PyTorch is used for device memory and streams: ``KiviCache`` allocates the caller-owned
cache buffers as torch tensors and passes their pointers.  The module raises ``KiviError`` if the
library is missing or a call fails; there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

PKG = os.path.dirname(os.path.abspath(__file__))
# KIVI_LIB=debug selects the debug build (libkivi_debug.so: device-side bounds checks); any other
# value is taken as the path of the library to load.
LIB_PATH = {"": os.path.join(PKG, "libkivi.so"), "debug": os.path.join(PKG, "libkivi_debug.so")}.get(
    os.environ.get("KIVI_LIB", ""), os.environ.get("KIVI_LIB", ""))

KIVI_OK = 0
STATUS_NAMES = {
    0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "CAPACITY", 4: "RESIDUAL_FULL",
    5: "RESIDUAL_NOT_FULL", 6: "EMPTY", 7: "WORKSPACE", 8: "CUDA", 9: "DEVICE_TIMEOUT", 10: "STATE",
    11: "INTERNAL",
}
BUFFERS = ("k_codes", "v_codes", "k_scale", "k_zero", "v_scale", "v_zero", "k_res", "v_res")


class KiviError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        self.code = STATUS_NAMES.get(status, str(status))
        super().__init__(f"{where}: {self.code}")


class kivi_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("batch", "num_kv_heads", "head_dim", "bits", "group_k", "group_v", "residual", "capacity",
                 "online_k", "fine_groups")]


class kivi_cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("k_zero", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("v_zero", ctypes.c_void_p),
                ("k_res", ctypes.c_void_p), ("v_res", ctypes.c_void_p),
                ("n_quant", ctypes.c_int32), ("n_res", ctypes.c_int32)]


class kivi_rotary(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("magnitude", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("turns", ctypes.c_uint64 * 64)]


class kivi_heads(ctypes.Structure):
    _fields_ = [("x_dev", ctypes.c_void_p), ("y_dev", ctypes.c_void_p), ("weight_dev", ctypes.c_void_p),
                ("num_heads", ctypes.c_int32), ("reserved", ctypes.c_int32)] + \
               [(n, ctypes.c_int64) for n in ("x_batch", "x_token", "x_head", "y_batch", "y_token", "y_head")]


_HEADS = struct.Struct("@PPPii6q")  # kivi_heads


class kivi_paged_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("num_pages", "num_seqs", "max_blocks", "num_kv_heads", "head_dim", "bits", "group_k", "group_v",
                 "residual")]


PAGED_BUFFERS = BUFFERS + ("block_table", "free_pages", "queue")


class kivi_paged_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in PAGED_BUFFERS]


class kivi_paged_plan(ctypes.Structure):
    _fields_ = [("cu_tokens", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("runs", ctypes.c_void_p),
                ("counts", ctypes.c_void_p), ("max_tokens", ctypes.c_int32), ("max_runs", ctypes.c_int32)]


DTYPE_F16, DTYPE_BF16 = 0, 1
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4}

_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libkivi.so (once).  Raises KiviError-like RuntimeError when it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} (run python -m bit_asymmetric_kv_02_b200.build)")
    lib = ctypes.CDLL(path)
    P, I32, U64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64, ctypes.c_size_t
    I64, F32, F64 = ctypes.c_int64, ctypes.c_float, ctypes.c_double
    cfgp, cachep = ctypes.POINTER(kivi_config), ctypes.POINTER(kivi_cache)
    pcfgp, pcachep, planp = (ctypes.POINTER(s) for s in (kivi_paged_config, kivi_paged_cache, kivi_paged_plan))
    rotp = ctypes.POINTER(kivi_rotary)
    sig = {
        "kivi_abi_version": (I32, []),
        "kivi_strerror": (ctypes.c_char_p, [I32]),
        "kivi_check_config": (I32, [cfgp]),
        "kivi_cache_sizes": (I32, [cfgp, ctypes.POINTER(SZ)]),
        "kivi_quantize_prefill": (I32, [cfgp, cachep, P, P, I32, P]),
        "kivi_quantize_prefill_prefix_k": (I32, [cfgp, cachep, P, P, I32, P]),
        "kivi_append_token": (I32, [cfgp, cachep, P, P, P]),
        "kivi_flush_residual": (I32, [cfgp, cachep, P]),
        "kivi_decode_workspace_bytes": (SZ, [cfgp, I32]),
        "kivi_decode_attention": (I32, [cfgp, cachep, P, I32, ctypes.c_float, P, P, SZ, P, P]),
        "kivi_append_decode_attention": (I32, [cfgp, cachep, P, P, P, I32, ctypes.c_float, P, P, SZ, P, P]),
        "kivi_decode_step": (I32, [cfgp, cachep, P, P, P, I32, ctypes.c_float, P, P, SZ, P, P]),
        "kivi_decode_attention_noalloc": (I32, [cfgp, cachep, P, I32, ctypes.c_float, P, P, P]),
        "kivi_window_workspace_bytes": (SZ, [cfgp, I32]),
        "kivi_decode_attention_window": (I32, [cfgp, cachep, P, I32, F32, I32, I32, P, P, SZ, P, P]),
        "kivi_rotary_init": (I32, [rotp, I32, I32, F64, I32, F64, F64, F64, I32]),
        "kivi_rotary_apply": (I32, [rotp, I32, I32, I32, P, I32, P, P, P, F32, P]),  # heads: kivi_heads or their bytes
        "kivi_paged_check_config": (I32, [pcfgp]),
        "kivi_paged_sizes": (I32, [pcfgp, ctypes.POINTER(SZ)]),
        "kivi_paged_build_tables": (I32, [pcfgp, pcachep, I32, P, P, P, P, planp, P, P]),
        "kivi_paged_append": (I32, [pcfgp, pcachep, planp, P, P, I64, I64, P, P]),
        "kivi_paged_workspace_bytes": (SZ, [pcfgp, I32]),
        "kivi_paged_decode_attention": (I32, [pcfgp, pcachep, I32, P, P, P, I32, I32, F32, I32, I32, P, P, SZ, P, P]),
        "kivi_paged_plan_attention": (I32, [pcfgp, pcachep, planp, I32, P, P, I32, I32, F32, I32, I32, P, P, SZ, P, P]),
        "kivi_read_status": (I32, [P, P]),
        "kivi_debug_inject": (I32, [I32, U64]),
        "kivi_debug_status": (I32, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    _lib = lib
    return lib


def _check(status: int, where: str) -> None:
    if status != KIVI_OK:
        raise KiviError(status, where)


# ---- C-ABI functions, same names ------------------------------------------------------------
def kivi_abi_version() -> int:
    return load_library().kivi_abi_version()


def kivi_strerror(status: int) -> str:
    return load_library().kivi_strerror(status).decode()


def kivi_check_config(cfg: kivi_config) -> int:
    return load_library().kivi_check_config(ctypes.byref(cfg))


def kivi_cache_sizes(cfg: kivi_config) -> list[int]:
    out = (ctypes.c_size_t * len(BUFFERS))()
    _check(load_library().kivi_cache_sizes(ctypes.byref(cfg), out), "kivi_cache_sizes")
    return list(out)


def kivi_quantize_prefill(cfg, cache, k_ptr: int, v_ptr: int, num_tokens: int, stream: int) -> None:
    _check(load_library().kivi_quantize_prefill(ctypes.byref(cfg), ctypes.byref(cache), k_ptr, v_ptr,
                                                num_tokens, stream), "kivi_quantize_prefill")


def kivi_quantize_prefill_prefix_k(cfg, cache, k_ptr: int, v_ptr: int, num_tokens: int, stream: int) -> None:
    _check(load_library().kivi_quantize_prefill_prefix_k(ctypes.byref(cfg), ctypes.byref(cache), k_ptr, v_ptr,
                                                         num_tokens, stream), "kivi_quantize_prefill_prefix_k")


def kivi_append_token(cfg, cache, k_new_ptr: int, v_new_ptr: int, stream: int) -> None:
    _check(load_library().kivi_append_token(ctypes.byref(cfg), ctypes.byref(cache), k_new_ptr, v_new_ptr,
                                            stream), "kivi_append_token")


def kivi_flush_residual(cfg, cache, stream: int) -> None:
    _check(load_library().kivi_flush_residual(ctypes.byref(cfg), ctypes.byref(cache), stream),
           "kivi_flush_residual")


def kivi_decode_workspace_bytes(cfg, num_q_heads: int) -> int:
    return load_library().kivi_decode_workspace_bytes(ctypes.byref(cfg), num_q_heads)


def kivi_decode_attention(cfg, cache, q_ptr: int, num_q_heads: int, scale: float, out_ptr: int,
                          ws_ptr: int, ws_bytes: int, status_ptr: int | None, stream: int) -> None:
    _check(load_library().kivi_decode_attention(ctypes.byref(cfg), ctypes.byref(cache), q_ptr, num_q_heads,
                                                scale, out_ptr, ws_ptr, ws_bytes, status_ptr, stream),
           "kivi_decode_attention")


def kivi_append_decode_attention(cfg, cache, k_new_ptr: int, v_new_ptr: int, q_ptr: int, num_q_heads: int,
                                 scale: float, out_ptr: int, ws_ptr: int, ws_bytes: int, status_ptr: int | None,
                                 stream: int) -> None:
    _check(load_library().kivi_append_decode_attention(ctypes.byref(cfg), ctypes.byref(cache), k_new_ptr, v_new_ptr,
                                                       q_ptr, num_q_heads, scale, out_ptr, ws_ptr, ws_bytes,
                                                       status_ptr, stream),
           "kivi_append_decode_attention")


def kivi_decode_step(cfg, cache, k_new_ptr: int, v_new_ptr: int, q_ptr: int, num_q_heads: int, scale: float,
                     out_ptr: int, ws_ptr: int, ws_bytes: int, status_ptr: int | None, stream: int) -> None:
    _check(load_library().kivi_decode_step(ctypes.byref(cfg), ctypes.byref(cache), k_new_ptr, v_new_ptr, q_ptr,
                                           num_q_heads, scale, out_ptr, ws_ptr, ws_bytes, status_ptr, stream),
           "kivi_decode_step")


def kivi_decode_attention_noalloc(cfg, cache, q_ptr: int, num_q_heads: int, scale: float, out_ptr: int,
                                  status_ptr: int | None, stream: int) -> None:
    """Decode attention with the library's fixed scratch array instead of a caller workspace, for
    callers that cannot allocate device memory at decode time (see include/kivi.h)."""
    _check(load_library().kivi_decode_attention_noalloc(ctypes.byref(cfg), ctypes.byref(cache), q_ptr, num_q_heads,
                                                        scale, out_ptr, status_ptr, stream),
           "kivi_decode_attention_noalloc")


def kivi_window_workspace_bytes(cfg, num_q_heads: int) -> int:
    return load_library().kivi_window_workspace_bytes(ctypes.byref(cfg), num_q_heads)


def kivi_decode_attention_window(cfg, cache, q_ptr: int, num_q_heads: int, scale: float, window: int, sinks: int,
                                 out_ptr: int, ws_ptr: int, ws_bytes: int, status_ptr: int | None, stream: int) -> None:
    _check(load_library().kivi_decode_attention_window(ctypes.byref(cfg), ctypes.byref(cache), q_ptr, num_q_heads,
                                                       scale, window, sinks, out_ptr, ws_ptr, ws_bytes, status_ptr,
                                                       stream), "kivi_decode_attention_window")


def kivi_rotary_init(rotary_dim: int, interleaved: int, theta: float, scaling: int, factor: float, low: float,
                     high: float, original_positions: int) -> kivi_rotary:
    r = kivi_rotary()
    _check(load_library().kivi_rotary_init(ctypes.byref(r), rotary_dim, interleaved, theta, scaling, factor, low, high,
                                           original_positions), "kivi_rotary_init")
    return r


def kivi_rotary_apply(rotary, dtype: int, batch: int, tokens: int, positions_ptr: int | None, position0: int, q, k, v,
                      eps: float, stream: int) -> None:
    """q, k, v: kivi_heads, the bytes of one, or None."""
    ref = [ctypes.byref(h) if isinstance(h, kivi_heads) else h for h in (q, k, v)]
    _check(load_library().kivi_rotary_apply(ctypes.byref(rotary), dtype, batch, tokens, positions_ptr, position0, *ref,
                                            eps, stream), "kivi_rotary_apply")


def kivi_paged_check_config(cfg: kivi_paged_config) -> int:
    return load_library().kivi_paged_check_config(ctypes.byref(cfg))


def kivi_paged_sizes(cfg: kivi_paged_config) -> list[int]:
    out = (ctypes.c_size_t * len(PAGED_BUFFERS))()
    _check(load_library().kivi_paged_sizes(ctypes.byref(cfg), out), "kivi_paged_sizes")
    return list(out)


def kivi_paged_build_tables(cfg, cache, num_rows: int, lens_ptr: int, new_tokens_ptr: int, lens_out_ptr: int,
                            queue_out_ptr: int, plan, status_ptr: int | None, stream: int) -> None:
    _check(load_library().kivi_paged_build_tables(ctypes.byref(cfg), ctypes.byref(cache), num_rows, lens_ptr,
                                                  new_tokens_ptr, lens_out_ptr, queue_out_ptr, ctypes.byref(plan),
                                                  status_ptr, stream), "kivi_paged_build_tables")


def kivi_paged_append(cfg, cache, plan, k_ptr: int, v_ptr: int, token_stride: int, head_stride: int,
                      status_ptr: int | None, stream: int) -> None:
    _check(load_library().kivi_paged_append(ctypes.byref(cfg), ctypes.byref(cache), ctypes.byref(plan), k_ptr, v_ptr,
                                            token_stride, head_stride, status_ptr, stream), "kivi_paged_append")


def kivi_paged_workspace_bytes(cfg, num_q_heads: int) -> int:
    return load_library().kivi_paged_workspace_bytes(ctypes.byref(cfg), num_q_heads)


def kivi_paged_decode_attention(cfg, cache, num_rows: int, lens_ptr: int, cu_tokens_ptr: int | None, q_ptr: int,
                                num_q_rows: int, num_q_heads: int, scale: float, window: int, sinks: int, out_ptr: int,
                                ws_ptr: int, ws_bytes: int, status_ptr: int | None, stream: int) -> None:
    _check(load_library().kivi_paged_decode_attention(ctypes.byref(cfg), ctypes.byref(cache), num_rows, lens_ptr,
                                                      cu_tokens_ptr, q_ptr, num_q_rows, num_q_heads, scale, window,
                                                      sinks, out_ptr, ws_ptr, ws_bytes, status_ptr, stream),
           "kivi_paged_decode_attention")


def kivi_paged_plan_attention(cfg, cache, plan, num_rows: int, lens_ptr: int, q_ptr: int, num_q_rows: int, num_q_heads: int,
                              scale: float, window: int, sinks: int, out_ptr: int, ws_ptr: int, ws_bytes: int,
                              status_ptr: int | None, stream: int) -> None:
    _check(load_library().kivi_paged_plan_attention(ctypes.byref(cfg), ctypes.byref(cache), ctypes.byref(plan), num_rows,
                                                    lens_ptr, q_ptr, num_q_rows, num_q_heads, scale, window, sinks, out_ptr,
                                                    ws_ptr, ws_bytes, status_ptr, stream),
           "kivi_paged_plan_attention")


def kivi_read_status(status_ptr: int, stream: int) -> int:
    return load_library().kivi_read_status(status_ptr, stream)


def kivi_debug_inject(mode: int, value: int = 0) -> None:
    _check(load_library().kivi_debug_inject(mode, value), "kivi_debug_inject")


def kivi_debug_status() -> int:
    """The first device-side check failure of the debug build since the last call (0: none)."""
    return load_library().kivi_debug_status()


# ---- torch-owned cache --------------------------------------------------------------------------
class KiviCache:
    """Caller-owned device buffers of one cache, allocated as torch tensors, plus the C struct.

    The arguments are the fields of kivi_config (include/kivi.h).  online_k: K rows are coded at
    append with the newest block's (s, z) once a block exists.  fine_groups: group_k counts tokens
    (one K pair per channel per group_k tokens) and group_v channels (one V pair per token per group_v
    channels).  num_q_heads sizes the decode workspace (default: one query head per KV head)."""

    def __init__(self, batch: int, num_kv_heads: int, capacity: int, bits: int = 2, group_k: int = 32,
                 group_v: int = 32, residual: int = 128, head_dim: int = 128, num_q_heads: int | None = None,
                 device=None, online_k: bool = False, fine_groups: bool = False):
        import torch
        self.torch = torch
        self.device = _device(torch, device)
        self.cfg = kivi_config(batch, num_kv_heads, head_dim, bits, group_k, group_v, residual, capacity,
                               1 if online_k else 0, 1 if fine_groups else 0)
        st = kivi_check_config(self.cfg)
        if st != KIVI_OK:
            raise KiviError(st, "kivi_check_config")
        sizes = kivi_cache_sizes(self.cfg)
        self.buffers = {}
        for name, nbytes in zip(BUFFERS, sizes):
            # uint8 storage padded to 16 bytes so an empty buffer still has an aligned pointer
            self.buffers[name] = torch.empty(max(16, nbytes), dtype=torch.uint8, device=self.device)
        self.c = kivi_cache(*[self.buffers[n].data_ptr() for n in BUFFERS], 0, 0)
        self.num_q_heads = num_q_heads or num_kv_heads
        self.ws_bytes = kivi_decode_workspace_bytes(self.cfg, self.num_q_heads)
        if self.ws_bytes == 0:
            raise KiviError(1, "kivi_decode_workspace_bytes")
        self.workspace = torch.zeros(self.ws_bytes + 256, dtype=torch.uint8, device=self.device)
        off = (-self.workspace.data_ptr()) % 256
        self.ws_ptr = self.workspace.data_ptr() + off
        self.status = torch.zeros(4, dtype=torch.int32, device=self.device)
        self._window_ws = {}
        self.index = self.status.device.index

    # views of the buffers in the layout of include/kivi.h
    def view(self, name: str):
        t = self.torch
        c = self.cfg
        B, H, C, d, R = c.batch, c.num_kv_heads, c.capacity, c.head_dim, c.residual
        P = 32 // c.bits
        shapes = {
            "k_codes": (t.int32, (B, H, C, d // P)), "v_codes": (t.int32, (B, H, C // P, d)),
            "k_scale": (t.float16, (B, H, C // R, d // c.group_k)), "k_zero": (t.float16, (B, H, C // R, d // c.group_k)),
            "v_scale": (t.float16, (B, H, C // c.group_v)), "v_zero": (t.float16, (B, H, C // c.group_v)),
            "k_res": (t.float16, (B, H, R, d)), "v_res": (t.float16, (B, H, R, d)),
        }
        if c.fine_groups:   # K: per channel per group_k tokens; V: per token per group_v channels
            for n_, sh in (("k_scale", (B, H, C // c.group_k, d)), ("k_zero", (B, H, C // c.group_k, d)),
                           ("v_scale", (B, H, C, d // c.group_v)), ("v_zero", (B, H, C, d // c.group_v))):
                shapes[n_] = (t.float16, sh)
        dtype, shape = shapes[name]
        n = math.prod(shape) * (4 if dtype == t.int32 else 2)
        return self.buffers[name][:n].view(dtype).view(shape)

    @property
    def n_quant(self) -> int:
        return self.c.n_quant

    @property
    def n_res(self) -> int:
        return self.c.n_res

    def _stream(self, stream) -> int:
        s = stream if stream is not None else self.torch.cuda.current_stream(self.device)
        return s.cuda_stream

    def prefill(self, k, v, stream=None) -> None:
        """k, v: contiguous fp16 device tensors [B][H][T][d]."""
        assert k.dtype == self.torch.float16 and k.is_contiguous() and v.is_contiguous()
        kivi_quantize_prefill(self.cfg, self.c, k.data_ptr(), v.data_ptr(), k.shape[2], self._stream(stream))

    def prefill_prefix_k(self, k, v, stream=None) -> None:
        """prefill with one K group over the whole quantized prefix (kivi_quantize_prefill_prefix_k)."""
        assert k.dtype == self.torch.float16 and k.is_contiguous() and v.is_contiguous()
        kivi_quantize_prefill_prefix_k(self.cfg, self.c, k.data_ptr(), v.data_ptr(), k.shape[2], self._stream(stream))

    def append(self, k_new, v_new, stream=None) -> None:
        """k_new, v_new: contiguous fp16 device tensors [B][H][d]."""
        kivi_append_token(self.cfg, self.c, k_new.data_ptr(), v_new.data_ptr(), self._stream(stream))

    def flush(self, stream=None) -> None:
        kivi_flush_residual(self.cfg, self.c, self._stream(stream))

    def attend(self, q, out=None, scale: float | None = None, stream=None, status: bool = True):
        """q: contiguous fp16 device tensor [B][Hq][d]; returns out (fp16, same shape)."""
        if out is None:
            out = self.torch.empty_like(q)
        scale = 1.0 / math.sqrt(self.cfg.head_dim) if scale is None else scale
        kivi_decode_attention(self.cfg, self.c, q.data_ptr(), q.shape[1], scale, out.data_ptr(), self.ws_ptr,
                              self.ws_bytes, self.status.data_ptr() if status else None, self._stream(stream))
        return out

    def append_attend(self, k_new, v_new, q, out=None, scale: float | None = None, stream=None,
                      status: bool = True):
        """append(k_new, v_new) then attend(q), in one kernel launch."""
        if out is None:
            out = self.torch.empty_like(q)
        scale = 1.0 / math.sqrt(self.cfg.head_dim) if scale is None else scale
        kivi_append_decode_attention(self.cfg, self.c, k_new.data_ptr(), v_new.data_ptr(), q.data_ptr(), q.shape[1],
                                     scale, out.data_ptr(), self.ws_ptr, self.ws_bytes,
                                     self.status.data_ptr() if status else None, self._stream(stream))
        return out

    def step(self, k_new, v_new, q, out=None, scale: float | None = None, stream=None, status: bool = True):
        """One streaming decode step: append(k_new, v_new), attend(q), and quantize the residual in
        the same launch when this token fills it (kivi_decode_step)."""
        if out is None:
            out = self.torch.empty_like(q)
        scale = 1.0 / math.sqrt(self.cfg.head_dim) if scale is None else scale
        kivi_decode_step(self.cfg, self.c, k_new.data_ptr(), v_new.data_ptr(), q.data_ptr(), q.shape[1], scale,
                         out.data_ptr(), self.ws_ptr, self.ws_bytes, self.status.data_ptr() if status else None,
                         self._stream(stream))
        return out

    def attend_window(self, q, window: int, sinks: int = 0, out=None, scale: float | None = None, stream=None,
                      status: bool = True):
        """attend(q) in which the newest token sees only the last `window` tokens (0: all) and the first
        `sinks` (kivi_decode_attention_window).  The workspace for a number of query heads is allocated
        and cleared on its first call, on the current stream: make that call before a capture."""
        _expect(self, "q", q, (self.cfg.batch, None, self.cfg.head_dim), self.torch.float16)
        hq = q.shape[1]
        ws = self._window_ws.get(hq)
        if ws is None:
            nbytes = kivi_window_workspace_bytes(self.cfg, hq)
            if nbytes == 0:
                raise KiviError(1, "kivi_window_workspace_bytes")
            ws = self._window_ws[hq] = _Workspace(self, nbytes, stream)
        out = _output(self, out, q, stream)
        scale = 1.0 / math.sqrt(self.cfg.head_dim) if scale is None else scale
        with _on(self):
            kivi_decode_attention_window(self.cfg, self.c, q.data_ptr(), hq, scale, _int32("window", window),
                                         _int32("sinks", sinks), out.data_ptr(), ws.ptr, ws.nbytes,
                                         self.status.data_ptr() if status else None, _raw_stream(self, stream))
        return out

    def step_rotary(self, rotary: "Rotary", k_new, v_new, q, q_weight=None, k_weight=None, eps: float = 1e-6, out=None,
                    scale: float | None = None, stream=None, status: bool = True):
        """step() with keys and queries as the projections give them: each head normed where it has a
        weight and rotated to the new token's position (Rotary.apply), then appended and attended.
        k_new, v_new, q: fp16 or bf16 [B][heads][128], of any strides that keep head rows whole; out fp16, as q."""
        for name, x, heads in (("q", q, None), ("k_new", k_new, self.cfg.num_kv_heads), ("v_new", v_new, self.cfg.num_kv_heads)):
            _expect(self, name, x, (self.cfg.batch, heads, self.cfg.head_dim), x.dtype, contiguous=False)
        v = None if v_new.dtype == self.torch.float16 and v_new.is_contiguous() else v_new.unsqueeze(2)
        q, k_new, v = rotary.apply(q.unsqueeze(2), k_new.unsqueeze(2), v, positions=self.n_quant + self.n_res,
                                   q_weight=q_weight, k_weight=k_weight, eps=eps, stream=stream)
        q, k_new, v_new = q.squeeze(2), k_new.squeeze(2), v_new if v is None else v.squeeze(2)
        return self.step(k_new, v_new, q, out=_output(self, out, q, stream), scale=scale, stream=stream, status=status)

    def read_status(self, stream=None) -> int:
        return kivi_read_status(self.status.data_ptr(), self._stream(stream))


# ---- argument checks and buffers of the torch layer ----------------------------------------------
def _expect(owner, name: str, t, shape, dtype, contiguous: bool = True) -> None:
    """Raises ValueError unless t is a tensor of that dtype and shape (None: any extent) on the owner's
    device, dense unless contiguous is False."""
    got = t.shape
    ok = t.dtype is dtype and len(got) == len(shape)
    if ok:
        for want, n in zip(shape, got):
            if want is not None and want != n:
                ok = False
    if not ok:
        raise ValueError(f"{name}: want {dtype} {list(shape)}, got {t.dtype} {list(got)}")
    if not t.is_cuda or t.get_device() != owner.index:
        raise ValueError(f"{name}: on {t.device}, the cache is on {owner.status.device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")


def _vector(owner, name: str, t, n, dtype) -> None:
    """_expect of one dimension (n None: any extent)."""
    if not (t.dtype is dtype and t.dim() == 1 and (n is None or t.shape[0] == n) and t.get_device() == owner.index
            and t.is_contiguous()):
        _expect(owner, name, t, (n,), dtype)


def _row_strides(t) -> tuple:
    """Strides of a [tokens][heads][128] tensor's first two dimensions; 0 where the extent leaves them without meaning."""
    (n, h, _), (a, b, _) = t.shape, t.stride()
    return a if n > 1 else 0, b if h > 1 else 0


def _raw_stream(owner, stream) -> int:
    """The handle of `stream`, or of the owner's device's current stream."""
    return stream.cuda_stream if stream is not None else owner.torch._C._cuda_getCurrentRawStream(owner.index)


def _device(torch, device):
    """torch.device(device); None: the current CUDA device."""
    return torch.device("cuda" if device is None else device)


class _Same:
    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_SAME = _Same()


def _on(owner):
    """A context on the owner's device, for free where it is the current one."""
    return _SAME if owner.index == owner.torch._C._cuda_getDevice() else owner.torch.cuda.device(owner.index)


def _int32(name: str, x: int) -> int:
    """x, which the C call takes as an int32 (ctypes would drop its upper bits)."""
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError(f"{name}: {x} is not an int32")
    return x


def _output(owner, out, q, stream):
    """`out`, checked, or a new tensor like q that belongs to the stream the call runs on."""
    if out is not None:
        _expect(owner, "out", out, q.shape, owner.torch.float16)
        return out
    if stream is None:
        return owner.torch.empty_like(q)
    with owner.torch.cuda.stream(stream):
        return owner.torch.empty_like(q)


class _Workspace:
    """A zeroed, 256-byte aligned workspace of its own, cleared on the stream that first uses it."""

    def __init__(self, owner, nbytes: int, stream=None):
        torch = owner.torch
        with torch.cuda.stream(stream):  # None: the current stream
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("the first call with a number of query heads allocates its workspace: make it before the capture")
            self.buffer = torch.zeros(nbytes + 256, dtype=torch.uint8, device=owner.device)
        self.ptr = self.buffer.data_ptr() + (-self.buffer.data_ptr()) % 256
        self.nbytes = nbytes


# ---- rotary positions and head norms -------------------------------------------------------------
class Rotary:
    """A position rotation with optional norms per head (kivi_rotary_init, kivi_rotary_apply).

    rotary_dim: leading channels of a head that rotate (a multiple of 16); interleaved: pairs (2 i, 2 i + 1)
    instead of (i, i + rotary_dim / 2); scaling: one of ROPE_SCALINGS with its factor and, for "bands" and
    "ramp", the turns low and high over original_positions (defaults: bands 1 and 4, ramp 1 and 32)."""

    def __init__(self, rotary_dim: int = 128, theta: float = 10000.0, interleaved: bool = False, scaling: str = "none",
                 factor: float = 1.0, low: float = 1.0, high: float | None = None, original_positions: int = 8192):
        import torch
        self.torch = torch
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling: one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
        if high is None:
            high = 32.0 if scaling == "ramp" else 4.0
        self.c = kivi_rotary_init(rotary_dim, 1 if interleaved else 0, theta, ROPE_SCALINGS[scaling], factor, low, high,
                                  original_positions)

    def _heads(self, name: str, x, y, weight, like, stream) -> tuple:
        """The bytes of kivi_heads of x ([tokens][heads][128], or [B][heads][T][128] as the cache's prefill
        takes it) and the output tensor."""
        torch = self.torch
        shape, wanted = x.shape, like.shape
        n = len(shape)
        if x is not like and (x.dtype is not like.dtype or not x.is_cuda or x.get_device() != like.get_device() or n != len(wanted)
                              or shape[0] != wanted[0] or (n == 4 and shape[2] != wanted[2])):
            raise ValueError(f"{name}: {x.dtype} {list(shape)} on {x.device} does not go with {like.dtype} {list(wanted)} on {like.device}")
        if shape[-1] != 128:
            raise ValueError(f"{name}: heads of {shape[-1]} channels, want 128")
        if y is None:
            if stream is None:
                y = torch.empty_like(x, dtype=torch.float16, memory_format=torch.contiguous_format)
            else:
                with torch.cuda.stream(stream):
                    y = torch.empty_like(x, dtype=torch.float16, memory_format=torch.contiguous_format)
        elif y.dtype is not torch.float16 or y.shape != shape or y.device != x.device:
            raise ValueError(f"{name} output: want float16 {list(shape)} on {x.device}")
        sx, sy = x.stride(), y.stride()
        if sx[-1] != 1 or sy[-1] != 1:
            raise ValueError(f"{name}: channels must be contiguous")
        if 0 in sy and any(m > 1 and s == 0 for m, s in zip(shape, sy)):
            raise ValueError(f"{name} output: expanded dimensions share memory")
        w = 0
        if weight is not None:
            if weight.dtype is not x.dtype or weight.shape != (128,) or weight.get_device() != x.get_device() or not weight.is_contiguous():
                raise ValueError(f"{name} weight: want contiguous {x.dtype} [128] on {x.device}")
            w = weight.data_ptr()
        if n == 4:
            return _HEADS.pack(x.data_ptr(), y.data_ptr(), w, shape[1], 0, sx[0], sx[2], sx[1], sy[0], sy[2], sy[1]), y
        return _HEADS.pack(x.data_ptr(), y.data_ptr(), w, shape[1], 0, 0, sx[0], sx[1], 0, sy[0], sy[1]), y

    def apply(self, q, k, v=None, positions=0, q_weight=None, k_weight=None, eps: float = 1e-6, q_out=None, k_out=None,
              v_out=None, stream=None):
        """Norms (where a weight is given) and rotates q and k, converts v, all to fp16, in one launch;
        returns (q, k, v), v None when it was not given.  Tensors are fp16 or bf16 [tokens][heads][128] or
        [B][heads][T][128], of any strides that keep head rows whole (slices of a fused projection).
        positions: int32 device tensor of one entry per token ([tokens] or [B][T]), or the first position.
        Outputs may be given; an fp16 input may be its own output."""
        call, outputs = self._arguments(q, k, v, positions, q_weight, k_weight, eps, q_out, k_out, v_out, stream)
        self._launch(*call)
        return outputs

    def _arguments(self, q, k, v, positions, q_weight, k_weight, eps, q_out, k_out, v_out, stream) -> tuple:
        """apply()'s checks: what _launch takes, and the outputs."""
        torch = self.torch
        dtype = DTYPE_F16 if q.dtype is torch.float16 else DTYPE_BF16
        n = q.dim()
        if (dtype == DTYPE_BF16 and q.dtype is not torch.bfloat16) or not q.is_cuda or n not in (3, 4):
            raise ValueError(f"q: want fp16 or bf16 [tokens][heads][128] or [B][heads][T][128] on the GPU, "
                             f"got {q.dtype} {list(q.shape)} on {q.device}")
        hq, q_out = self._heads("q", q, q_out, q_weight, q, stream)
        hk, k_out = self._heads("k", k, k_out, k_weight, q, stream)
        hv = None
        if v is not None:
            hv, v_out = self._heads("v", v, v_out, None, q, stream)
        batch, tokens = (q.shape[0], q.shape[2]) if n == 4 else (1, q.shape[0])
        index = q.get_device()
        if isinstance(positions, int):
            ptr, first = None, _int32("positions", positions)
        else:
            if positions.dtype is not torch.int32 or positions.numel() != batch * tokens or not positions.is_contiguous() \
                    or positions.get_device() != index:
                raise ValueError(f"positions: want contiguous int32 of {batch * tokens} entries on {q.device}")
            ptr, first = positions.data_ptr(), 0
        s = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(index)
        return (index, batch, tokens, (self.c, dtype, batch, tokens, ptr, first, hq, hk, hv, eps, s)), (q_out, k_out, v_out)

    def _launch(self, index: int, batch: int, tokens: int, args: tuple) -> None:
        if batch * tokens == 0:
            return
        call = load_library().kivi_rotary_apply
        if index == self.torch._C._cuda_getDevice():
            st = call(*args)
        else:
            with self.torch.cuda.device(index):
                st = call(*args)
        _check(st, "kivi_rotary_apply")

    @staticmethod
    def _check_rules(args: tuple) -> None:
        """The library's checks of what _arguments packed that are not made there."""
        bad, heads = not 0.0 <= args[9] <= 3.0e38, 0
        for packed in args[6:9]:
            if packed is not None:
                x, y, w, n, _, a, b, c, d, e, f = _HEADS.unpack(packed)
                bad = bad or (x | y | w) & 15 or (a | b | c | d | e | f) & 7
                heads += n
        if bad or heads > 1 << 20:
            raise KiviError(1 if bad else 2, "kivi_rotary_apply")


# ---- torch-owned paged cache ---------------------------------------------------------------------
class PagedPlan:
    """One step's tables (kivi_paged_plan): cu_tokens [num_seqs + 1], positions [max_tokens], runs
    [max_runs][8] and counts [2] as int32 tensors."""

    def __init__(self, cache: "PagedKiviCache", max_tokens: int):
        torch = cache.torch
        runs = 2 * cache.cfg.num_seqs + max_tokens // cache.cfg.residual
        if max_tokens < 1 or runs >= 1 << 31:
            raise ValueError(f"max_tokens: {max_tokens}")
        self.cu_tokens = torch.zeros(cache.cfg.num_seqs + 1, dtype=torch.int32, device=cache.device)
        self.positions = torch.zeros(max_tokens, dtype=torch.int32, device=cache.device)
        self.runs = torch.zeros(runs, 8, dtype=torch.int32, device=cache.device)
        self.counts = torch.zeros(2, dtype=torch.int32, device=cache.device)
        self.max_tokens = max_tokens
        self.num_seqs, self.residual = cache.cfg.num_seqs, cache.cfg.residual
        self.c = kivi_paged_plan(self.cu_tokens.data_ptr(), self.positions.data_ptr(), self.runs.data_ptr(),
                                 self.counts.data_ptr(), max_tokens, runs)
        self.max_runs = runs
        self._narrow = max_tokens, self.c

    def of(self, rows: int) -> kivi_paged_plan:
        """The plan, for `rows` tokens at most: none may lie past the rows that a call has."""
        if rows >= self.max_tokens:
            return self.c
        last, c = self._narrow
        if last != rows:
            a = self.c
            c = kivi_paged_plan(a.cu_tokens, a.positions, a.runs, a.counts, rows, a.max_runs)
            self._narrow = rows, c
        return c


class PagedKiviCache:
    """Caller-owned device buffers of a paged cache (include/kivi.h) as torch tensors, for sequences of
    different lengths that come and go.  A step:

        plan = cache.new_plan(max_tokens)                    # once
        cache.build_tables(plan, lens, new_tokens)           # tables, positions, slot map; lens advanced
        q, k, v = rotary.apply(q, k, v, positions=plan.positions[:tokens])
        cache.append(plan, k, v)
        out = cache.attend(lens, q, plan=plan)               # the newest token of every sequence

    or all four as step().  The layers of a model share one set of tables: PagedKiviCache(..., tables=first) for
    the others, one build_tables() a step, and append() and attend() with that plan in every layer.
    Everything a step reads or advances is on the device, so it can be captured in a CUDA graph and replayed
    (make one uncaptured attend() with its number of query heads first).  Calls of one cache that overlap on
    the GPU are not allowed: they share buffers and workspaces."""

    def __init__(self, num_pages: int, num_seqs: int, max_blocks: int, num_kv_heads: int, bits: int = 2, group_k: int = 32,
                 group_v: int = 32, residual: int = 128, head_dim: int = 128, num_q_heads: int | None = None, device=None,
                 tables: "PagedKiviCache | None" = None):
        import torch
        self.torch = torch
        self.device = tables.device if tables is not None and device is None else _device(torch, device)
        self.cfg = kivi_paged_config(num_pages, num_seqs, max_blocks, num_kv_heads, head_dim, bits, group_k, group_v,
                                     residual)
        st = kivi_paged_check_config(self.cfg)
        if st != KIVI_OK:
            raise KiviError(st, "kivi_paged_check_config")
        shared = ()
        if tables is not None:  # a layer whose blocks lie where the other one's do
            mine, other = self.cfg, tables.cfg
            if (mine.num_pages, mine.num_seqs, mine.max_blocks, mine.residual) != \
                    (other.num_pages, other.num_seqs, other.max_blocks, other.residual):
                raise ValueError("tables: of a cache with other pages, sequences or blocks")
            shared = PAGED_BUFFERS[len(BUFFERS):]
        self.buffers = {}
        for name, nbytes in zip(PAGED_BUFFERS, kivi_paged_sizes(self.cfg)):
            self.buffers[name] = tables.buffers[name] if name in shared else \
                torch.empty(max(16, nbytes), dtype=torch.uint8, device=self.device)
        self.device = self.buffers["k_codes"].device
        if self.device != self.buffers["queue"].device:
            raise ValueError(f"tables: on {tables.device}, the cache on {self.device}")
        self.c = kivi_paged_cache(*[self.buffers[n].data_ptr() for n in PAGED_BUFFERS])
        if not shared:
            self.view("block_table").fill_(-1)
            self.view("free_pages").copy_(torch.arange(num_pages, dtype=torch.int32))
            self.view("queue").copy_(torch.tensor([0, num_pages]))
        self.status = torch.zeros(4, dtype=torch.int32, device=self.device)
        self.index = self.status.device.index
        self.num_seqs, self.residual, self.kv_heads, self.head_dim = num_seqs, residual, num_kv_heads, head_dim
        self._ws = {}
        if num_q_heads is not None:
            self._workspace(num_q_heads, None)

    def _workspace(self, num_q_heads: int, stream) -> _Workspace:
        ws = self._ws.get(num_q_heads)
        if ws is None:
            nbytes = kivi_paged_workspace_bytes(self.cfg, num_q_heads)
            if nbytes == 0:
                raise KiviError(1, "kivi_paged_workspace_bytes")
            ws = self._ws[num_q_heads] = _Workspace(self, nbytes, stream)
        return ws

    def _call(self, fn, *args) -> None:
        with _on(self):
            fn(self.cfg, self.c, *args)

    def _check_plan(self, plan: PagedPlan) -> None:
        if plan.num_seqs != self.num_seqs or plan.residual != self.residual or plan.counts.get_device() != self.index:
            raise ValueError(f"plan: of {plan.num_seqs} sequences and {plan.residual}-token blocks on {plan.counts.device}")

    def view(self, name: str):
        """The buffer in the layout of include/kivi.h."""
        t, c = self.torch, self.cfg
        N, S, H, R, d, P = c.num_pages, c.num_seqs, c.num_kv_heads, c.residual, c.head_dim, 32 // c.bits
        dtype, shape = {
            "k_codes": (t.int32, (N, H, R, d // P)), "v_codes": (t.int32, (N, H, R // P, d)),
            "k_scale": (t.float16, (N, H, d // c.group_k)), "k_zero": (t.float16, (N, H, d // c.group_k)),
            "v_scale": (t.float16, (N, H, R // c.group_v)), "v_zero": (t.float16, (N, H, R // c.group_v)),
            "k_res": (t.float16, (S, H, R, d)), "v_res": (t.float16, (S, H, R, d)),
            "block_table": (t.int32, (S, c.max_blocks)), "free_pages": (t.int32, (N,)), "queue": (t.int64, (2,)),
        }[name]
        n = math.prod(shape) * dtype.itemsize
        return self.buffers[name][:n].view(dtype).view(shape)

    def new_plan(self, max_tokens: int) -> PagedPlan:
        """Buffers for steps of at most max_tokens new tokens."""
        return PagedPlan(self, max_tokens)

    def build_tables(self, plan: PagedPlan, lens, new_tokens, lens_out=None, queue_out=None, stream=None,
                     status: bool = True) -> None:
        """Tables of a step (kivi_paged_build_tables): lens, new_tokens int32 [n], n <= num_seqs.  The new
        lengths and queue replace the old ones unless lens_out (int32 [n]) or queue_out (int64 [2]) take them."""
        self._call(*self._tables_call(plan, plan.c, lens, new_tokens, lens_out, queue_out, stream, status))

    def _tables_call(self, plan, c, lens, new_tokens, lens_out, queue_out, stream, status) -> tuple:
        """build_tables()' checks: the arguments of _call.  c: the plan, or one of fewer tokens in its buffers."""
        self._check_plan(plan)
        i32, n = self.torch.int32, lens.shape[0] if lens.dim() == 1 else None
        _vector(self, "lens", lens, n, i32)
        _vector(self, "new_tokens", new_tokens, n, i32)
        if lens_out is not None:
            _vector(self, "lens_out", lens_out, n, i32)
        if queue_out is not None:
            _vector(self, "queue_out", queue_out, 2, self.torch.int64)
        return (kivi_paged_build_tables, n, lens.data_ptr(), new_tokens.data_ptr(),
                (lens if lens_out is None else lens_out).data_ptr(),
                self.c.queue if queue_out is None else queue_out.data_ptr(), c,
                self.status.data_ptr() if status else None, _raw_stream(self, stream))

    def append(self, plan: PagedPlan, k, v, stream=None, status: bool = True) -> None:
        """Writes a step's tokens (kivi_paged_append): k, v fp16 [tokens][H][128] of equal strides that keep
        head rows whole, tokens at least the plan's count (a plan of more: KIVI_ERR_INTERNAL in the status word)."""
        self._check_plan(plan)
        self._call(*self._append_call(plan, k, v, stream, status))

    def _append_call(self, plan, k, v, stream, status) -> tuple:
        """append()'s checks: the arguments of _call."""
        f16, shape = self.torch.float16, k.shape
        _expect(self, "k", k, (None, self.kv_heads, self.head_dim), f16, contiguous=False)
        if v.shape != shape or v.dtype is not f16 or v.get_device() != self.index:
            _expect(self, "v", v, shape, f16, contiguous=False)
        strides, other = k.stride(), v.stride()
        if strides != other or strides[2] != 1:
            strides = _row_strides(k)
            if shape[0] > 0 and (strides != _row_strides(v) or k.stride(2) != 1 or other[2] != 1):
                raise ValueError(f"k, v: strides {k.stride()} and {other}; want equal strides and contiguous channels")
        return (kivi_paged_append, plan.of(shape[0]), k.data_ptr(), v.data_ptr(), strides[0], strides[1],
                self.status.data_ptr() if status else None, _raw_stream(self, stream))

    def attend(self, lens, q, plan: PagedPlan | None = None, out=None, scale: float | None = None, window: int = 0,
               sinks: int = 0, stream=None, status: bool = True):
        """Attention of the newest token of each sequence (kivi_paged_decode_attention): lens int32 [n], q
        fp16 [rows][Hq][128].  Without a plan row i is sequence i; with one (kivi_paged_plan_attention), q holds
        a row per new token of the step, and only the last of each sequence that the tables could serve is
        attended.  Other rows of out stay as they are: give `out` or do not read them."""
        call, out = self._attend_call(lens, q, plan, out, scale, window, sinks, stream, status)
        if q.shape[0] > 0:
            self._call(*call)
        return out

    def _attend_call(self, lens, q, plan, out, scale, window, sinks, stream, status) -> tuple:
        """attend()'s checks: the arguments of _call, and the output."""
        _vector(self, "lens", lens, None, self.torch.int32)
        _expect(self, "q", q, (None, None, self.head_dim), self.torch.float16)
        if plan is not None:
            self._check_plan(plan)
        elif q.shape[0] < lens.shape[0]:
            raise ValueError(f"q: {q.shape[0]} rows for {lens.shape[0]} sequences")
        ws = self._workspace(q.shape[1], stream)
        out = _output(self, out, q, stream)
        n, heads, _ = q.shape
        rest = (q.data_ptr(), n, heads, 1.0 / math.sqrt(self.head_dim) if scale is None else scale, _int32("window", window),
                _int32("sinks", sinks), out.data_ptr(), ws.ptr, ws.nbytes, self.status.data_ptr() if status else None,
                _raw_stream(self, stream))
        if plan is None:
            return (kivi_paged_decode_attention, lens.shape[0], lens.data_ptr(), None, *rest), out
        return (kivi_paged_plan_attention, plan.c, lens.shape[0], lens.data_ptr(), *rest), out

    def step(self, plan: PagedPlan, lens, new_tokens, q, k, v, rotary: Rotary | None = None, q_weight=None, k_weight=None,
             eps: float = 1e-6, out=None, scale: float | None = None, window: int = 0, sinks: int = 0, stream=None,
             status: bool = True):
        """A step of a layer: tables, norms and rotation (with a rotary), append, attention; lens advances.
        q, k, v: [tokens][heads][128], fp16 (with a rotary: or bf16), packed by sequence; new_tokens sums to
        their rows or fewer: of more, nothing is planned and KIVI_ERR_CAPACITY reported in the status word.
        Returns the attention output [tokens][Hq][128] (rows: see attend).  A step that raises has changed
        nothing: every argument is checked before the first launch."""
        f16, turn = self.torch.float16, None
        if q.shape[0] > plan.max_tokens:
            raise ValueError(f"q: {q.shape[0]} rows, the plan holds {plan.max_tokens}")
        if q.dim() != 3 or k.dim() != 3 or v.dim() != 3 or q.get_device() != self.index:
            raise ValueError(f"q, k, v: want [tokens][heads][128] on {self.status.device}, got {list(q.shape)} on {q.device}, "
                             f"{list(k.shape)}, {list(v.shape)}")
        if rotary is not None:
            turn, (q, k, v16) = rotary._arguments(q, k, v if v.dtype is not f16 else None, plan.positions[:q.shape[0]], q_weight, k_weight,
                                                  eps, None, None, None, stream)
            rotary._check_rules(turn[3])
            v = v if v16 is None else v16
        apart = k.stride() != v.stride() and _row_strides(k) != _row_strides(v)
        if apart or not q.is_contiguous():
            with self.torch.cuda.stream(stream):  # None: the current stream
                if apart:
                    k, v = k if turn is not None else k.contiguous(), v.contiguous()  # rotated keys are dense, and not there yet
                q = q.contiguous()
        append = self._append_call(plan, k, v, stream, status)
        rows = min(q.shape[0], k.shape[0])
        tables = self._tables_call(plan, plan.of(max(rows, 1)), lens, new_tokens, None, None, stream, status)
        attend, out = self._attend_call(lens, q, plan, out, scale, window, sinks, stream, status)
        # the library's own checks, of calls behind the first
        if (append[2] | append[3]) & 15 or (append[4] | append[5]) & 7:
            raise KiviError(1, "kivi_paged_append")
        if min(plan.max_runs, k.shape[0]) * self.kv_heads > 0x7fffffff:
            raise KiviError(2, "kivi_paged_append")
        if (attend[4] | attend[10]) & 15 or window < 0 or sinks < 0 or not abs(attend[7]) <= 3.0e38:
            raise KiviError(1, "kivi_paged_plan_attention")
        with _on(self):
            tables[0](self.cfg, self.c, *tables[1:])
            if turn is not None:
                rotary._launch(*turn)
            append[0](self.cfg, self.c, *append[1:])
            if q.shape[0] > 0:
                attend[0](self.cfg, self.c, *attend[1:])
        return out

    def read_status(self, stream=None) -> int:
        return kivi_read_status(self.status.data_ptr(), _raw_stream(self, stream))

"""Thin ctypes binding of ``libtq.so`` (the C ABI declared in include/tq.h).

The functions below carry the C names and only marshal arguments; every
step of the compressed-cache path runs in the library's CUDA kernels.
PyTorch is used for device memory and streams only (``TQCache``).  There is
no fallback: if the library is missing, loading raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from ctypes import (POINTER, Structure, c_char_p, c_float, c_int8, c_int32, c_int64,
                    c_size_t, c_uint8, c_uint16, c_uint64, c_void_p)

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libtq.so")

TQ_OK = 0
STATUS_NAMES = {0: "TQ_OK", 1: "TQ_ERR_INVALID_ARG", 2: "TQ_ERR_UNSUPPORTED",
                3: "TQ_ERR_CAPACITY", 4: "TQ_ERR_RANGE", 5: "TQ_ERR_TIMEOUT",
                6: "TQ_ERR_CUDA"}
TOKENS_PER_BLOCK = 64


class TQError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS_NAMES.get(code, code)}")
        self.code = code


class tq_config(Structure):
    _fields_ = [("batch", c_int32), ("num_q_heads", c_int32), ("num_kv_heads", c_int32),
                ("head_dim", c_int32), ("hot_window", c_int32), ("cold_capacity", c_int64),
                ("b_r", c_int32), ("b_theta", c_int32), ("qjl_bits", c_int32),
                ("seed", c_uint64)]


class tq_vec_config(Structure):
    _fields_ = [("dim", c_int32), ("b_r", c_int32), ("b_theta", c_int32), ("qjl_bits", c_int32),
                ("seed", c_uint64)]


class tq_q8_cache(Structure):
    _fields_ = [("batch", c_int32), ("num_kv_heads", c_int32), ("head_dim", c_int32), ("format", c_int32),
                ("dtype", c_int32), ("capacity", c_int64), ("k_codes", c_void_p), ("v_codes", c_void_p),
                ("k_scales", c_void_p), ("v_scales", c_void_p), ("k_recent", c_void_p),
                ("v_recent", c_void_p), ("status", c_void_p)]


_lib = None

# (name, restype, argtypes) of every exported symbol
SIGNATURES = [
    ("tq_status_string", c_char_p, [c_int32]),
    ("tq_abi_version", c_int32, []),
    ("tq_cache_bytes", c_int32, [POINTER(tq_config), POINTER(c_size_t), POINTER(c_size_t),
                                 POINTER(c_size_t)]),
    ("tq_cache_create", c_int32, [POINTER(tq_config), c_void_p, c_void_p, c_void_p, c_void_p,
                                  POINTER(c_void_p)]),
    ("tq_cache_destroy", c_int32, [c_void_p]),
    ("tq_cache_counts", c_int32, [c_void_p, POINTER(c_int64), POINTER(c_int32), POINTER(c_int32)]),
    ("tq_encode_append", c_int32, [c_void_p, c_void_p, c_void_p, c_int64, c_void_p]),
    ("tq_encode_append_rows", c_int32, [c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_void_p]),
    ("tq_evict_window_rows", c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p]),
    ("tq_cache_row_counts", c_int32, [c_void_p, c_int32, POINTER(c_int64), POINTER(c_int32),
                                      POINTER(c_int32)]),
    ("tq_evict_window", c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_void_p]),
    ("tq_decode_attention", c_int32, [c_void_p, c_void_p, c_void_p, c_float, c_void_p]),
    ("tq_decode_attention_static", c_int32, [c_void_p, c_void_p, c_void_p, c_float, c_void_p]),
    ("tq_decode_attention_gated", c_int32, [c_void_p, c_void_p, c_void_p, c_float, c_float, c_void_p,
                                            c_void_p]),
    ("tq_tc_bytes", c_int32, [POINTER(tq_config), POINTER(c_size_t)]),
    ("tq_tc_enable", c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    ("tq_get_status", c_int32, [c_void_p, c_void_p]),
    ("tq_set_attend_events", c_int32, [c_void_p, c_void_p, c_void_p]),
    ("tq_set_wait_limit", c_int32, [c_void_p, c_int64]),
    ("tq_promotion_bytes", c_int32, [POINTER(tq_config), POINTER(c_size_t)]),
    ("tq_promotion_enable", c_int32, [c_void_p, c_void_p, c_float, c_int32, c_void_p]),
    ("tq_promotion_state", c_int32, [c_void_p, c_void_p, c_void_p]),
    ("tq_export_cold", c_int32, [c_void_p, c_int32, c_int32, c_int64, c_int64, c_void_p,
                                 c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    ("tq_vec_bytes", c_int32, [POINTER(tq_vec_config), c_int64, c_int32, POINTER(c_size_t),
                               POINTER(c_size_t)]),
    ("tq_vec_create", c_int32, [POINTER(tq_vec_config), c_int64, c_int32, c_void_p, c_void_p,
                                POINTER(c_void_p)]),
    ("tq_vec_destroy", c_int32, [c_void_p]),
    ("tq_encode_vectors", c_int32, [c_void_p, c_void_p, c_int64, c_int64, c_void_p, c_void_p]),
    ("tq_ip_search", c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_void_p,
                               c_void_p]),
    ("tq_vec_get_status", c_int32, [c_void_p, c_void_p]),
    ("tq_export_vectors", c_int32, [c_void_p, c_void_p, c_int64, c_int64, c_void_p, c_void_p,
                                    c_void_p, c_void_p, c_void_p]),
    ("tq_q8_append", c_int32, [c_void_p, c_char_p, c_void_p]),
    ("tq_q8_read", c_int32, [c_void_p, c_void_p, c_int64, c_int32, c_void_p, c_void_p, c_void_p]),
    ("tq_q8_attention_bytes", c_int32, [c_void_p, c_int32, c_int32, POINTER(c_size_t)]),
    ("tq_q8_attention", c_int32, [c_void_p, c_char_p, c_void_p]),
    ("tq_q8_get_status", c_int32, [c_void_p, c_void_p]),
    ("tq_qk_norm_rope", c_int32, [c_char_p, c_void_p]),
    ("tq_rotation_signs", c_int32, [c_uint64, c_int32, POINTER(c_int8)]),
    ("tq_qjl_matrix", c_int32, [c_uint64, c_int32, c_int32, POINTER(c_float)]),
]


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; build it with "
                               "`python -m compressed_decode_attention_encode_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, res, args in SIGNATURES:
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(code: int, what: str) -> None:
    if code != TQ_OK:
        raise TQError(code, what)


def make_config(batch, num_q_heads, num_kv_heads, head_dim, hot_window, cold_capacity,
                b_r, b_theta, qjl_bits, seed=0) -> tq_config:
    return tq_config(batch, num_q_heads, num_kv_heads, head_dim, hot_window, cold_capacity,
                     b_r, b_theta, qjl_bits, seed)


# ---- functions with the C names -------------------------------------------

def tq_status_string(code: int) -> str:
    return lib().tq_status_string(code).decode()


def tq_abi_version() -> int:
    return lib().tq_abi_version()


def tq_cache_bytes(cfg: tq_config):
    h, c, w = c_size_t(), c_size_t(), c_size_t()
    _check(lib().tq_cache_bytes(ctypes.byref(cfg), ctypes.byref(h), ctypes.byref(c),
                                ctypes.byref(w)), "tq_cache_bytes")
    return h.value, c.value, w.value


def tq_cache_create(cfg: tq_config, hot_ptr: int, cold_ptr: int, ws_ptr: int, stream: int) -> int:
    out = c_void_p()
    _check(lib().tq_cache_create(ctypes.byref(cfg), hot_ptr, cold_ptr, ws_ptr, stream,
                                 ctypes.byref(out)), "tq_cache_create")
    return out.value


def tq_cache_destroy(handle: int) -> None:
    _check(lib().tq_cache_destroy(handle), "tq_cache_destroy")


def tq_cache_counts(handle: int):
    nc, nh, rp = c_int64(), c_int32(), c_int32()
    _check(lib().tq_cache_counts(handle, ctypes.byref(nc), ctypes.byref(nh), ctypes.byref(rp)),
           "tq_cache_counts")
    return nc.value, nh.value, rp.value


def tq_encode_append(handle: int, k_ptr: int, v_ptr: int, n: int, stream: int) -> None:
    _check(lib().tq_encode_append(handle, k_ptr, v_ptr, n, stream), "tq_encode_append")


def tq_evict_window(handle: int, k_ptr: int, v_ptr: int, n: int, stream: int) -> None:
    _check(lib().tq_evict_window(handle, k_ptr, v_ptr, n, stream), "tq_evict_window")


def tq_decode_attention(handle: int, q_ptr: int, out_ptr: int, scale: float, stream: int) -> None:
    _check(lib().tq_decode_attention(handle, q_ptr, out_ptr, scale, stream), "tq_decode_attention")


def tq_decode_attention_static(handle: int, q_ptr: int, out_ptr: int, scale: float,
                               stream: int) -> None:
    _check(lib().tq_decode_attention_static(handle, q_ptr, out_ptr, scale, stream),
           "tq_decode_attention_static")


def tq_decode_attention_gated(handle: int, q_ptr: int, out_ptr: int, scale: float, threshold: float,
                              head_skip_ptr, stream: int) -> None:
    _check(lib().tq_decode_attention_gated(handle, q_ptr, out_ptr, scale, threshold, head_skip_ptr,
                                           stream), "tq_decode_attention_gated")


def tq_tc_bytes(cfg: tq_config) -> int:
    n = c_size_t()
    _check(lib().tq_tc_bytes(ctypes.byref(cfg), ctypes.byref(n)), "tq_tc_bytes")
    return n.value


def tq_tc_enable(handle: int, tc_ptr: int, lam, eta, gate, stream: int) -> None:
    def arr(x):
        a = np.ascontiguousarray(np.asarray(x, dtype=np.float32))
        return a, a.ctypes.data_as(c_void_p)
    la, lp = arr(lam)
    ea, ep = arr(eta)
    ga, gp = arr(gate)
    _check(lib().tq_tc_enable(handle, tc_ptr, lp, ep, gp, stream), "tq_tc_enable")


def tq_get_status(handle: int, stream: int) -> int:
    return lib().tq_get_status(handle, stream)


def tq_set_attend_events(handle: int, start: int, stop: int) -> None:
    _check(lib().tq_set_attend_events(handle, start, stop), "tq_set_attend_events")


def tq_promotion_bytes(cfg: tq_config) -> int:
    n = c_size_t()
    _check(lib().tq_promotion_bytes(ctypes.byref(cfg), ctypes.byref(n)), "tq_promotion_bytes")
    return n.value


def tq_promotion_enable(handle: int, mem_ptr: int, threshold: float, sticky: int, stream: int) -> None:
    _check(lib().tq_promotion_enable(handle, mem_ptr, threshold, sticky, stream), "tq_promotion_enable")


def tq_set_wait_limit(handle: int, limit_ns: int) -> None:
    _check(lib().tq_set_wait_limit(handle, limit_ns), "tq_set_wait_limit")


def tq_rotation_signs(seed: int, d: int) -> np.ndarray:
    out = np.empty(d, dtype=np.int8)
    _check(lib().tq_rotation_signs(seed, d, out.ctypes.data_as(POINTER(c_int8))),
           "tq_rotation_signs")
    return out


def tq_qjl_matrix(seed: int, m: int, d: int) -> np.ndarray:
    out = np.empty((m, d), dtype=np.float32)
    _check(lib().tq_qjl_matrix(seed, m, d, out.ctypes.data_as(POINTER(c_float))), "tq_qjl_matrix")
    return out


# ---- device-memory plumbing (PyTorch) --------------------------------------

def _stream_handle(stream=None) -> int:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _ptr(t) -> int:
    return t.data_ptr()


class TQCache:
    """A per-layer compressed cache: PyTorch-allocated device buffers bound to
    a library handle.  Every method is a direct call into libtq.so."""

    def __init__(self, cfg: tq_config, device="cuda", stream=None):
        import torch
        self.cfg = cfg
        self.device = torch.device(device)
        hot, cold, ws = tq_cache_bytes(cfg)
        self.hot = torch.empty(max(hot, 256), dtype=torch.uint8, device=self.device)
        self.cold = torch.empty(max(cold, 256), dtype=torch.uint8, device=self.device)
        self.ws = torch.empty(max(ws, 256), dtype=torch.uint8, device=self.device)
        self.bytes = dict(hot=hot, cold=cold, workspace=ws)
        self.handle = tq_cache_create(cfg, _ptr(self.hot), _ptr(self.cold), _ptr(self.ws),
                                      _stream_handle(stream))

    def close(self):
        if getattr(self, "handle", None):
            tq_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # shape checks are the library's; these only guard the Python objects
    @staticmethod
    def _dev16(t):
        import torch
        if t.dtype != torch.float16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("expected a contiguous CUDA float16 tensor")
        return _ptr(t)

    def encode_append(self, k, v, stream=None):
        n = k.shape[2]
        tq_encode_append(self.handle, self._dev16(k), self._dev16(v), n, _stream_handle(stream))

    def evict_window(self, k_new, v_new, stream=None):
        tq_evict_window(self.handle, self._dev16(k_new), self._dev16(v_new), k_new.shape[2],
                        _stream_handle(stream))

    def decode_attention(self, q, out=None, softmax_scale=0.0, stream=None):
        import torch
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        if out.dtype != torch.float32 or not out.is_contiguous():
            raise ValueError("out must be contiguous float32")
        tq_decode_attention(self.handle, self._dev16(q), _ptr(out), softmax_scale,
                            _stream_handle(stream))
        return out

    def decode_attention_gated(self, q, threshold, out=None, head_skip=None, softmax_scale=0.0,
                               stream=None):
        """Decode attention whose cold tier is read only by the query heads
        whose largest hot score q.k is below ``threshold``; ``head_skip``
        (int32 [B, Hq] on the device) receives 1 for the heads that skipped."""
        import torch
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        if out.dtype != torch.float32 or not out.is_contiguous():
            raise ValueError("out must be contiguous float32")
        hs = None
        if head_skip is not None:
            if head_skip.dtype != torch.int32 or not head_skip.is_cuda or not head_skip.is_contiguous():
                raise ValueError("head_skip must be a contiguous CUDA int32 tensor")
            hs = _ptr(head_skip)
        tq_decode_attention_gated(self.handle, self._dev16(q), _ptr(out), softmax_scale,
                                  float(threshold), hs, _stream_handle(stream))
        return out

    def enable_tensor_cache(self, lam, eta, gate, stream=None):
        """Switch evictions to the Tensor Cache tier: lam, eta per kv head,
        gate (g, before the sigmoid) per query head.  Returns the view of A
        [B, Hkv, d, d] (float32, on the device)."""
        import torch
        c = self.cfg
        if len(lam) != c.num_kv_heads or len(eta) != c.num_kv_heads or len(gate) != c.num_q_heads:
            raise ValueError("lam, eta: one per kv head; gate: one per query head")
        self.tc_mem = torch.empty(tq_tc_bytes(c), dtype=torch.uint8, device=self.device)
        tq_tc_enable(self.handle, _ptr(self.tc_mem), lam, eta, gate, _stream_handle(stream))
        n = c.batch * c.num_kv_heads * c.head_dim * c.head_dim
        return self.tc_mem[: 4 * n].view(torch.float32).view(c.batch, c.num_kv_heads, c.head_dim,
                                                             c.head_dim)

    def get_status(self, stream=None) -> int:
        return tq_get_status(self.handle, _stream_handle(stream))

    def set_attend_events(self, start=None, stop=None):
        """Record torch.cuda.Events around the attention kernel of the next
        decode calls (None, None stops recording)."""
        tq_set_attend_events(self.handle, start.cuda_event if start is not None else None,
                             stop.cuda_event if stop is not None else None)

    def enable_promotion(self, threshold=0.15, sticky=3, stream=None):
        """Attention-weighted promotion (sticky counters) on this handle;
        the library's buffer comes from PyTorch."""
        import torch
        self.promo_mem = torch.empty(tq_promotion_bytes(self.cfg), dtype=torch.uint8, device=self.device)
        tq_promotion_enable(self.handle, _ptr(self.promo_mem), float(threshold), int(sticky),
                            _stream_handle(stream))

    def promotion_state(self, stream=None):
        """Per (row, kv head): dict of counted positions -> counts, the
        promoted positions not yet moved, and the ring position."""
        units = self.cfg.batch * self.cfg.num_kv_heads
        out = np.zeros((units, 28), dtype=np.int32)
        _check(lib().tq_promotion_state(self.handle, out.ctypes.data, _stream_handle(stream)),
               "tq_promotion_state")
        res = []
        for u in range(units):
            o = out[u]
            res.append(dict(counts={int(o[4 + i]): int(o[12 + i]) for i in range(o[0])},
                            pending=[int(x) for x in o[20:20 + o[1]]], ring_pos=int(o[2])))
        return res

    def set_wait_limit(self, limit_ns: int):
        """Bounded-wait limit of the attention kernel (ns; 0 forces a
        timeout at the first wait, < 0 restores the default)."""
        tq_set_wait_limit(self.handle, limit_ns)

    def counts(self):
        return tq_cache_counts(self.handle)

    def row_counts(self, row: int):
        nc, nh, rp = c_int64(), c_int32(), c_int32()
        _check(lib().tq_cache_row_counts(self.handle, row, ctypes.byref(nc), ctypes.byref(nh),
                                         ctypes.byref(rp)), "tq_cache_row_counts")
        return nc.value, nh.value, rp.value

    def encode_append_rows(self, k, v, n_rows, stream=None):
        """Row b appends its first n_rows[b] tokens of k, v [B, Hkv, n_max, d]."""
        rows = np.ascontiguousarray(np.asarray(n_rows, dtype=np.int32))
        _check(lib().tq_encode_append_rows(self.handle, self._dev16(k), self._dev16(v), k.shape[2],
                                           rows.ctypes.data, _stream_handle(stream)),
               "tq_encode_append_rows")

    def evict_window_rows(self, k_new, v_new, n_rows, stream=None):
        """Row b inserts its first n_rows[b] tokens of k_new, v_new [B, Hkv, n_max, d]."""
        rows = np.ascontiguousarray(np.asarray(n_rows, dtype=np.int32))
        _check(lib().tq_evict_window_rows(self.handle, self._dev16(k_new), self._dev16(v_new),
                                          k_new.shape[2], rows.ctypes.data, _stream_handle(stream)),
               "tq_evict_window_rows")

    def hot_ring(self):
        """Views of the fp16 hot rings K, V: [B, Hkv, W, d] (slot order)."""
        import torch
        c = self.cfg
        n = c.batch * c.num_kv_heads * c.hot_window * c.head_dim
        h = self.hot[: 4 * n].view(torch.float16)
        shape = (c.batch, c.num_kv_heads, c.hot_window, c.head_dim)
        return h[:n].view(shape), h[n:].view(shape)

    def export_cold(self, row: int, kv_head: int, start: int, count: int, stream=None):
        """Canonical records of cold tokens start..start+count (host numpy)."""
        c = self.cfg
        kc = c.head_dim // 2 * (c.b_r + c.b_theta) // 8
        sg = c.qjl_bits // 8
        out = dict(k_codes=np.zeros((count, kc), np.uint8), k_bits=np.zeros((count, sg), np.uint8),
                   k_s16=np.zeros(count, np.uint16), k_rn16=np.zeros(count, np.uint16),
                   v_codes=np.zeros((count, kc), np.uint8), v_s16=np.zeros(count, np.uint16))
        p = {k: v.ctypes.data for k, v in out.items()}
        _check(lib().tq_export_cold(self.handle, row, kv_head, start, count, p["k_codes"],
                                    p["k_bits"], p["k_s16"], p["k_rn16"], p["v_codes"], p["v_s16"],
                                    _stream_handle(stream)), "tq_export_cold")
        return out


# ---- vector search ----------------------------------------------------------

def tq_vec_bytes(cfg: tq_vec_config, n: int, max_queries: int):
    c, w = c_size_t(), c_size_t()
    _check(lib().tq_vec_bytes(ctypes.byref(cfg), n, max_queries, ctypes.byref(c), ctypes.byref(w)),
           "tq_vec_bytes")
    return c.value, w.value


class TQVecIndex:
    """Compressed vector database + search handle (device memory from
    PyTorch; every method is a direct call into libtq.so)."""

    def __init__(self, dim, n, b_r=4, b_theta=4, qjl_bits=200, seed=0, max_queries=1024,
                 device="cuda", stream=None):
        import torch
        self.cfg = tq_vec_config(dim, b_r, b_theta, qjl_bits, seed)
        self.n = n
        cb, wb = tq_vec_bytes(self.cfg, n, max_queries)
        self.codes = torch.empty(max(cb, 256), dtype=torch.uint8, device=device)
        self.ws = torch.empty(max(wb, 256), dtype=torch.uint8, device=device)
        out = c_void_p()
        _check(lib().tq_vec_create(ctypes.byref(self.cfg), n, max_queries, self.ws.data_ptr(),
                                   _stream_handle(stream), ctypes.byref(out)), "tq_vec_create")
        self.handle = out.value

    def close(self):
        if getattr(self, "handle", None):
            _check(lib().tq_vec_destroy(self.handle), "tq_vec_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def encode(self, x, start=0, stream=None):
        """x: contiguous CUDA float32 [count, dim] -> database rows start.."""
        import torch
        if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
            raise ValueError("expected a contiguous CUDA float32 tensor")
        _check(lib().tq_encode_vectors(self.handle, x.data_ptr(), start, x.shape[0],
                                       self.codes.data_ptr(), _stream_handle(stream)),
               "tq_encode_vectors")

    def search(self, q, k=10, stream=None):
        """q: contiguous CUDA float32 [nq, dim] -> (scores [nq, k], idx [nq, k])."""
        import torch
        if q.dtype != torch.float32 or not q.is_cuda or not q.is_contiguous():
            raise ValueError("expected a contiguous CUDA float32 tensor")
        nq = q.shape[0]
        scores = torch.empty((nq, k), dtype=torch.float32, device=q.device)
        idx = torch.empty((nq, k), dtype=torch.int32, device=q.device)
        _check(lib().tq_ip_search(self.handle, self.codes.data_ptr(), q.data_ptr(), nq, k,
                                  scores.data_ptr(), idx.data_ptr(), _stream_handle(stream)),
               "tq_ip_search")
        return scores, idx

    def get_status(self, stream=None):
        """Latched device status of the searches (0 = TQ_OK); clears it."""
        return lib().tq_vec_get_status(self.handle, _stream_handle(stream))

    def export(self, start, count, stream=None):
        d = 64
        while d < self.cfg.dim:
            d *= 2
        kc = d // 2 * (self.cfg.b_r + self.cfg.b_theta) // 8
        mb = self.cfg.qjl_bits // 8
        out = dict(codes=np.zeros((count, kc), np.uint8), bits=np.zeros((count, mb), np.uint8),
                   s16=np.zeros(count, np.uint16), rn16=np.zeros(count, np.uint16))
        p = {k: v.ctypes.data for k, v in out.items()}
        _check(lib().tq_export_vectors(self.handle, self.codes.data_ptr(), start, count, p["codes"],
                                       p["bits"], p["s16"], p["rn16"], _stream_handle(stream)),
               "tq_export_vectors")
        return out


# ---- 8-bit cache ------------------------------------------------------------

# The argument structs tq_q8_append_args, tq_q8_attention_args and
# tq_qk_norm_rope_args as bytes: one packing costs a tenth of as many ctypes
# conversions (2.8 us less for the norm and rotation's 22).
_APPEND_ARGS = struct.Struct("@PP6qi4xPP").pack
_ATTENTION_ARGS = struct.Struct("@P3q2iPPf4xPPN").pack
_NORM_ROPE_ARGS = struct.Struct("@6iP3qP3q4Pfi2P").pack

Q8_BLOCK = 64        # tokens that share a scale
Q8_RING = 128        # slots of the 16-bit ring


def _q8_dtypes():
    import torch
    return {torch.float16: 0, torch.bfloat16: 1}


_torch = None        # the module, once a call has needed it

# Attention scratch by (device, stream): a stream's calls follow one another,
# whatever cache or thread they come from, so the layers of a model share it.
_scratch = {}


def _raw_stream(torch, index: int, stream) -> int:
    """The stream to launch on: ``stream``, or PyTorch's current one of the
    device.  The device must be the current one (the library launches there)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if stream.device.index != index:
        raise ValueError(f"expected a stream of cuda:{index}")
    return stream.cuda_stream


class TQ8Cache:
    """A layer's KV cache in 8 bits: whole blocks of 64 tokens as int8 or e4m3
    codes with one float32 scale per (row, kv head, block), the open block in a
    16-bit ring.  Every method is a direct call into libtq.so.

    The object keeps no lengths: each call takes ``lens``, an int32 tensor [B]
    on the cache's device, which the caller advances once per step for all
    layers, so that calls can be captured in CUDA graphs.  Host threads may call
    at the same time; what one call writes and another reads is ordered by
    their streams.

    A row may be set back (rejected drafts) to 64 tokens below the greatest
    length it has had, or to any multiple of 64, from which that counts anew.

    ``buffers``: tensors of an earlier cache to take over, by the names
    ``k_codes``, ``v_codes`` [B, Hkv, capacity, d] (int8 or float8_e4m3fn),
    ``k_scales``, ``v_scales`` [B, Hkv, capacity / 64] (float32), ``k_recent``,
    ``v_recent`` [B, Hkv, 128, d] (``dtype``)."""

    FORMATS = {"int8": 0, "e4m3": 1}

    def __init__(self, batch, num_kv_heads, head_dim, capacity, format="int8", dtype=None,
                 device="cuda", buffers=None):
        import torch
        self._torch = torch
        dtype = torch.float16 if dtype is None else dtype
        if format not in self.FORMATS:
            raise ValueError("format is 'int8' or 'e4m3'")
        if dtype not in _q8_dtypes():
            raise ValueError("dtype is torch.float16 or torch.bfloat16")
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.device, self.dtype = device, dtype
        code = torch.int8 if format == "int8" else torch.float8_e4m3fn
        shape = (batch, num_kv_heads)
        for kv in "kv":
            for name, more, dt in (("codes", (capacity, head_dim), code),
                                   ("scales", (capacity // Q8_BLOCK,), torch.float32),
                                   ("recent", (Q8_RING, head_dim), dtype)):
                t = buffers[f"{kv}_{name}"] if buffers is not None else None
                if t is None:
                    t = torch.empty(shape + more, dtype=dt, device=device)
                elif tuple(t.shape) != shape + more or t.dtype != dt or t.device != device or not t.is_contiguous():
                    raise ValueError(f"{kv}_{name}: expected a contiguous {dt} {list(shape + more)} on {device}")
                setattr(self, f"{kv}_{name}", t)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.struct = tq_q8_cache(batch, num_kv_heads, head_dim, self.FORMATS[format], _q8_dtypes()[dtype],
                                  capacity, _ptr(self.k_codes), _ptr(self.v_codes), _ptr(self.k_scales),
                                  _ptr(self.v_scales), _ptr(self.k_recent), _ptr(self.v_recent),
                                  _ptr(self.status))
        self._ref = ctypes.addressof(self.struct)
        self._lib = lib()
        self._index = device.index if device.type == "cuda" else -1
        self._shape = (batch, num_kv_heads, head_dim)
        self._scratch_size = {}
        # the sizes are checked here once, by the library (no device call)
        _check(self._lib.tq_q8_append(self._ref, _APPEND_ARGS(*[0] * 11), None), "TQ8Cache")

    def _on_device(self, method, *args):
        with self._torch.cuda.device(self.device):
            return method(*args)

    def _elsewhere(self):
        """Whether another device is the current one: the library launches there."""
        if self._index < 0:
            raise ValueError("the cache is not on a CUDA device")
        return self._torch._C._cuda_getDevice() != self._index

    def _ints(self, t, what):
        if t.dtype is not self._torch.int32 or t.get_device() != self._index or t.shape != self._shape[:1] \
                or not t.is_contiguous():
            raise ValueError(f"{what}: expected a contiguous int32 [{self._shape[0]}] on {self.device}")
        return t.data_ptr()

    def _values(self, t, what):
        if t.dtype is not self.dtype or t.get_device() != self._index:
            raise ValueError(f"{what}: expected {self.dtype} on {self.device}")
        s = t.stride()
        if s[-1] != 1:
            raise ValueError(f"{what}: the head dimension must be contiguous")
        return t.data_ptr(), s

    def append(self, k, v, lens, n_rows=None, stream=None):
        """k, v [B, Hkv, n, d] (any strides with d contiguous) become tokens
        lens[b] .. lens[b] + n_rows[b] - 1 of row b (n_rows None: n each)."""
        b, h, d = self._shape
        shape = k.shape
        if len(shape) != 4 or shape[0] != b or shape[1] != h or shape[3] != d or v.shape != shape:
            raise ValueError(f"k, v: expected [{b}, {h}, n, {d}]")
        kp, ks = self._values(k, "k")
        vp, vs = self._values(v, "v")
        lp = self._ints(lens, "lens")
        rp = 0 if n_rows is None else self._ints(n_rows, "n_rows")
        if self._elsewhere():
            return self._on_device(self.append, k, v, lens, n_rows, stream)
        args = _APPEND_ARGS(kp, vp, ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], shape[2], lp, rp)
        code = self._lib.tq_q8_append(self._ref, args, _raw_stream(self._torch, self._index, stream))
        if code:
            _check(code, "tq_q8_append")

    def read(self, lens, start=0, n=None, out=None, stream=None):
        """Positions start .. start + n - 1 of every row as 16-bit K, V
        [B, Hkv, n, d].  ``out``: a pair to write into, whose values that belong
        to no token stay; without it they are zero."""
        b, h, d = self._shape
        if out is None:
            if n is None:
                raise ValueError("read needs n or out")
            if stream is not None:                       # what is allocated here belongs to the call's stream
                with self._torch.cuda.stream(stream):
                    return self.read(lens, start, n)
            out = tuple(self._torch.zeros((b, h, n, d), dtype=self.dtype, device=self.device) for _ in "kv")
        ko, vo = out
        shape = ko.shape
        if len(shape) != 4 or shape[0] != b or shape[1] != h or shape[3] != d or vo.shape != shape \
                or (n is not None and n != shape[2]) or not ko.is_contiguous() or not vo.is_contiguous():
            raise ValueError(f"out: expected two contiguous [{b}, {h}, n, {d}]")
        kp, vp = self._values(ko, "out")[0], self._values(vo, "out")[0]
        lp = self._ints(lens, "lens")
        if self._elsewhere():
            return self._on_device(self.read, lens, start, n, out, stream)
        code = self._lib.tq_q8_read(self._ref, lp, start, shape[2], kp, vp,
                                    _raw_stream(self._torch, self._index, stream))
        if code:
            _check(code, "tq_q8_read")
        return out

    def scratch_bytes(self, num_q_heads, n):
        """Bytes of scratch of an attention call (as tq_q8_attention_bytes)."""
        key = (num_q_heads, n)
        size = self._scratch_size.get(key)
        if size is None:
            if self._elsewhere():
                return self._on_device(self.scratch_bytes, num_q_heads, n)
            got = c_size_t()
            _check(self._lib.tq_q8_attention_bytes(self._ref, num_q_heads, n, ctypes.byref(got)),
                   "tq_q8_attention_bytes")
            size = self._scratch_size[key] = got.value
        return size

    def _take_scratch(self, size, raw):
        """Scratch of the call: one buffer per stream, for all caches; a
        captured call gets its own, from its graph's memory, since graphs may be
        replayed beside anything."""
        torch = self._torch
        if torch._C._cuda_isCurrentStreamCapturing():
            return torch.empty(size, dtype=torch.uint8, device=self.device)
        key = self._index, raw
        t = _scratch.get(key)
        if t is None or t.shape[0] < size:
            t = _scratch[key] = torch.empty(size, dtype=torch.uint8, device=self.device)
        return t

    def attention(self, q, lens, n_rows=None, out=None, softmax_scale=0.0, scratch=None, stream=None):
        """q [B, n, Hq, d] (or [B, Hq, d] for one token): the newest n tokens'
        queries, attending to their row's positions up to their own; lens
        counts them.  Returns ``out`` in q's shape and type.  ``scratch``: a
        uint8 tensor of scratch_bytes for the call (without it the stream's)."""
        torch = self._torch
        if stream is not None:                           # what is allocated here belongs to the call's stream
            if stream.device != self.device:
                raise ValueError(f"expected a stream of {self.device}")
            with torch.cuda.stream(stream):
                return self.attention(q, lens, n_rows, out, softmax_scale, scratch)
        b, h, d = self._shape
        shape = q.shape
        dims = len(shape)
        if not 3 <= dims <= 4 or shape[0] != b or shape[-1] != d:
            raise ValueError(f"q: expected [{b}, n, Hq, {d}]")
        n, hq = (shape[1], shape[2]) if dims == 4 else (1, shape[1])
        index = self._index
        if q.dtype is not self.dtype or q.get_device() != index:
            raise ValueError(f"q: expected {self.dtype} on {self.device}")
        qs = q.stride()
        if qs[-1] != 1:
            raise ValueError("q: the head dimension must be contiguous")
        lp = self._ints(lens, "lens")
        rp = 0 if n_rows is None else self._ints(n_rows, "n_rows")
        if self._elsewhere():
            return self._on_device(self.attention, q, lens, n_rows, out, softmax_scale, scratch)
        raw = torch._C._cuda_getCurrentRawStream(index)
        key = hq, n
        size = self._scratch_size.get(key)
        if size is None:
            size = self.scratch_bytes(hq, n)
        if out is None:
            out = torch.empty(shape, dtype=self.dtype, device=self.device)
        elif out.shape != shape or out.dtype is not self.dtype or out.get_device() != index \
                or not out.is_contiguous():
            raise ValueError("out: expected a contiguous tensor of q's shape and type")
        if scratch is None:
            scratch = self._take_scratch(size, raw)
        elif scratch.dtype is not torch.uint8 or scratch.get_device() != index or not scratch.is_contiguous():
            raise ValueError(f"scratch: expected a contiguous uint8 tensor on {self.device}")
        args = _ATTENTION_ARGS(q.data_ptr(), qs[0], qs[1] if dims == 4 else 0, qs[-2], hq, n, lp, rp, softmax_scale,
                               out.data_ptr(), scratch.data_ptr(), scratch.shape[0])
        code = self._lib.tq_q8_attention(self._ref, args, raw)
        if code:
            _check(code, "tq_q8_attention")
        return out

    def get_status(self, stream=None):
        """Latched device status (0 = TQ_OK); waits for the stream, then clears it."""
        if self._elsewhere():
            return self._on_device(self.get_status, stream)
        return self._lib.tq_q8_get_status(self._ref, _raw_stream(self._torch, self._index, stream))


def qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                 q_out=None, k_out=None, stream=None):
    """Norm of every query and key head and rotation by position (see
    tq_qk_norm_rope): q [B, n, Hq, d], k [B, n, Hkv, d] (any strides with d
    contiguous, e.g. slices of a packed projection), positions int32 [B, n],
    inv_freq float32 [d / 2].  Returns q_out [B, n, Hq, d] and k_out
    [B, Hkv, n, d], the layouts that the caches' calls take."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    torch = _torch
    if stream is not None:                               # what is allocated here belongs to the call's stream
        if stream.device != q.device:
            raise ValueError(f"expected a stream of {q.device}")
        with torch.cuda.stream(stream):
            return qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, q_out, k_out)
    qs, ks, dtype, index = q.shape, k.shape, q.dtype, q.get_device()
    code = 0 if dtype is torch.float16 else 1 if dtype is torch.bfloat16 else -1
    if len(qs) != 4 or len(ks) != 4 or qs[:2] != ks[:2] or qs[3] != ks[3] or code < 0 or k.dtype is not dtype \
            or index < 0 or k.get_device() != index:
        raise ValueError("expected q [B, n, Hq, d] and k [B, n, Hkv, d], CUDA float16 or bfloat16 of one type and device")
    b, n, hq, d = qs
    hk = ks[2]
    s0, s1, s2, s3 = q.stride()
    t0, t1, t2, t3 = k.stride()
    if (s3 != 1 and q.numel()) or (t3 != 1 and k.numel()):
        raise ValueError("q, k: the head dimension must be contiguous")
    if q_out is None:
        q_out = torch.empty((b, n, hq, d), dtype=dtype, device=q.device)
    elif q_out.dtype is not dtype or q_out.shape != qs or q_out.get_device() != index or not q_out.is_contiguous():
        raise ValueError(f"q_out: expected a contiguous {dtype} {list(qs)} on cuda:{index}")
    if k_out is None:
        k_out = torch.empty((b, hk, n, d), dtype=dtype, device=q.device)
    elif k_out.dtype is not dtype or k_out.shape != (b, hk, n, d) or k_out.get_device() != index \
            or not k_out.is_contiguous():
        raise ValueError(f"k_out: expected a contiguous {dtype} {[b, hk, n, d]} on cuda:{index}")
    if positions.dtype is not torch.int32 or positions.shape != (b, n) or positions.get_device() != index \
            or not positions.is_contiguous():
        raise ValueError(f"positions: expected a contiguous int32 {[b, n]} on cuda:{index}")
    if inv_freq.dtype is not torch.float32 or inv_freq.shape != (d // 2,) or inv_freq.get_device() != index \
            or not inv_freq.is_contiguous():
        raise ValueError(f"inv_freq: expected a contiguous float32 {[d // 2]} on cuda:{index}")
    if q_weight is None:
        q_weight = 0
    else:
        if q_weight.dtype is not dtype or q_weight.shape != (d,) or q_weight.get_device() != index \
                or not q_weight.is_contiguous():
            raise ValueError(f"q_weight: expected a contiguous {dtype} {[d]} on cuda:{index}")
        q_weight = q_weight.data_ptr()
    if k_weight is None:
        k_weight = 0
    else:
        if k_weight.dtype is not dtype or k_weight.shape != (d,) or k_weight.get_device() != index \
                or not k_weight.is_contiguous():
            raise ValueError(f"k_weight: expected a contiguous {dtype} {[d]} on cuda:{index}")
        k_weight = k_weight.data_ptr()
    args = _NORM_ROPE_ARGS(b, n, hq, hk, d, code, q.data_ptr(), s0, s1, s2, k.data_ptr(), t0, t1, t2, positions.data_ptr(),
                           inv_freq.data_ptr(), q_weight, k_weight, eps, 1 if interleaved else 0, q_out.data_ptr(),
                           k_out.data_ptr())
    if torch._C._cuda_getDevice() == index:
        code = lib().tq_qk_norm_rope(args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            code = lib().tq_qk_norm_rope(args, torch._C._cuda_getCurrentRawStream(index))
    if code:
        _check(code, "tq_qk_norm_rope")
    return q_out, k_out

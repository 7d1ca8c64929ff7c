"""ctypes binding of libdosa (include/dosa.h).

Argument marshalling only: tensors become device pointers, the current torch
stream becomes the cudaStream_t, status codes become exceptions.  Every step of
the indexer runs in the library's CUDA kernels; there is no CPU fallback, and
loading fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdosa.so")

DOSA_BF16, DOSA_FP8_E4M3, DOSA_FP16 = 0, 1, 2
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported configuration",
          3: "workspace too small", 4: "CUDA error", 5: "device wait timed out",
          6: "device bounds check failed"}

# Every function the public header declares (the CPU tests check the export).
EXPORTS = ("dosa_index_config_default", "dosa_index_create", "dosa_index_destroy",
           "dosa_index_workspace_size", "dosa_index_topk", "dosa_index_dense_topk",
           "dosa_index_scores", "dosa_reference_scores", "dosa_index_certificate",
           "dosa_index_dense_topk_static", "dosa_topk_rows", "dosa_check_device",
           "dosa_status_string", "dosa_profile_enable", "dosa_profile_reset",
           "dosa_profile_read", "dosa_index_topk_host", "dosa_index_host_workspace_size",
           "dosa_index_decode_topk", "dosa_index_decode_workspace_size",
           "dosa_attn_config_default", "dosa_attn_create", "dosa_attn_destroy",
           "dosa_attn_prompt", "dosa_attn_prompt_workspace_size", "dosa_cache4_append",
           "dosa_cache4_read", "dosa_cache4_attend", "dosa_cache4_attend_workspace_size",
           "dosa_cache4_evict")
KERNELS = {"score": 0, "topk": 1, "reference": 2, "key_prep": 3, "cert_setup": 4,
           "certified": 5, "select": 6, "filter": 7, "decode": 8,
           "fill": 9, "block": 10, "rescore": 11, "rank": 12, "prompt": 13, "cache": 14,
           "attend": 15, "evict": 16}


class DosaError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)} ({code})")
        self.code = code


class Config(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int), ("d", ctypes.c_int), ("dtype", ctypes.c_int),
                ("max_K", ctypes.c_int), ("seed_first", ctypes.c_int),
                ("seed_last", ctypes.c_int), ("r", ctypes.c_int), ("G", ctypes.c_int),
                ("margin_log2", ctypes.c_int), ("screening", ctypes.c_int),
                ("sparse_writeback", ctypes.c_int), ("block_bound", ctypes.c_int),
                ("probe_sample", ctypes.c_int), ("short_dense_keys", ctypes.c_int)]


class Stats(ctypes.Structure):
    _fields_ = [("visible_pairs", ctypes.c_int64), ("seed_pairs", ctypes.c_int64),
                ("screened_pairs", ctypes.c_int64), ("rejected_pairs", ctypes.c_int64),
                ("exact_pairs", ctypes.c_int64), ("candidates", ctypes.c_int64),
                ("filtered_pairs", ctypes.c_int64), ("block_skipped_pairs", ctypes.c_int64),
                ("rescored_pairs", ctypes.c_int64), ("repaired_rows", ctypes.c_int64),
                ("rescreened_pairs", ctypes.c_int64)]

    def as_dict(self) -> dict:
        return {name: int(getattr(self, name)) for name, _ in self._fields_}


class AttnConfig(ctypes.Structure):
    _fields_ = [("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("d", ctypes.c_int),
                ("dtype", ctypes.c_int), ("scale", ctypes.c_float)]


class Rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class Cache4Arrays(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_params", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_params", ctypes.c_void_p),
                ("weight", ctypes.c_void_p), ("capacity", ctypes.c_int64)]


_lib = None
_P, _I, _I64, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t


def load(path: str = LIB_PATH):
    """Load libdosa.so and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built: run `python -m exact_certified_top_b200.build`")
    lib = ctypes.CDLL(path)
    lib.dosa_index_config_default.argtypes = [ctypes.POINTER(Config)]
    lib.dosa_index_config_default.restype = None
    lib.dosa_index_create.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(_P)]
    lib.dosa_index_destroy.argtypes = [_P]
    lib.dosa_index_destroy.restype = None
    lib.dosa_index_workspace_size.argtypes = [_P, _I64, _I64, _I, _I, _I64,
                                              ctypes.POINTER(_SZ)]
    common = [_P, _P, _P, _P, _P, _P, _P, _I, _I, _P, _P, _SZ, _P]
    lib.dosa_index_topk.argtypes = common + [ctypes.POINTER(Stats)]
    lib.dosa_index_dense_topk.argtypes = common
    lib.dosa_index_topk_host.argtypes = common + [ctypes.POINTER(Stats)]
    lib.dosa_index_decode_topk.argtypes = [_P, _P, _P, _P, _P, _P, _P, _I, _I, _P, _P, _P, _SZ,
                                           _P, ctypes.POINTER(Stats)]
    lib.dosa_index_decode_workspace_size.argtypes = [_P, _I64, _I64, _I, ctypes.POINTER(_SZ)]
    lib.dosa_index_host_workspace_size.argtypes = [_P, _I64, _I64, _I64, _I, _I64,
                                                   ctypes.POINTER(_SZ)]
    lib.dosa_index_scores.argtypes = [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _I64,
                                      _P, _P]
    lib.dosa_reference_scores.argtypes = [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P,
                                          _I64, _P]
    lib.dosa_index_dense_topk_static.argtypes = [_P, _P, _P, _P, _P, _P, _P, _I, _I, _P, _P]
    lib.dosa_index_certificate.argtypes = [_P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P, _SZ,
                                           _P]
    lib.dosa_topk_rows.argtypes = [_P, _I64, _P, _I64, _I, _P, _P]
    lib.dosa_check_device.argtypes = [_P, _P]
    rows, cache = ctypes.POINTER(Rows), ctypes.POINTER(Cache4Arrays)
    lib.dosa_attn_config_default.argtypes = [ctypes.POINTER(AttnConfig)]
    lib.dosa_attn_config_default.restype = None
    lib.dosa_attn_create.argtypes = [ctypes.POINTER(AttnConfig), ctypes.POINTER(_P)]
    lib.dosa_attn_destroy.argtypes = [_P]
    lib.dosa_attn_destroy.restype = None
    lib.dosa_attn_prompt.argtypes = [_P, rows, rows, rows, _P, _I, rows, _P, _P, _SZ, _P]
    lib.dosa_attn_prompt_workspace_size.argtypes = [_P, _P, _I, ctypes.POINTER(_SZ)]
    lib.dosa_cache4_append.argtypes = [_P, cache, rows, rows, _P, _I, _P]
    lib.dosa_cache4_read.argtypes = [_P, cache, _P, _I, rows, rows, _P]
    lib.dosa_cache4_attend.argtypes = [_P, cache, rows, _P, _I, _P, _I, _I, rows, _P, _P, _SZ, _P]
    lib.dosa_cache4_attend_workspace_size.argtypes = [_P, _P, _I, _I, _I, ctypes.POINTER(_SZ)]
    lib.dosa_cache4_evict.argtypes = [_P, cache, cache, _P, _I, _I64, _I64, _P, _I64, _P]
    lib.dosa_profile_enable.argtypes = [_I]
    lib.dosa_profile_reset.argtypes = []
    lib.dosa_profile_read.argtypes = [_I, ctypes.POINTER(_I64), ctypes.POINTER(ctypes.c_double)]
    lib.dosa_status_string.argtypes = [_I]
    lib.dosa_status_string.restype = ctypes.c_char_p
    for fn in EXPORTS:
        f = getattr(lib, fn)
        if f.restype is ctypes.c_int and fn not in ("dosa_index_config_default",):
            f.restype = ctypes.c_int
    _lib = lib
    return lib


def _check(fn: str, code: int):
    if code != 0:
        raise DosaError(fn, code)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The current stream's handle without building a Stream object, where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev=None):
    if _raw_stream is not None:
        return ctypes.c_void_p(_raw_stream(torch.cuda.current_device() if dev is None else dev))
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _seq_offsets(seq_offsets) -> torch.Tensor:
    so = torch.as_tensor(seq_offsets, dtype=torch.int64).cpu().contiguous()
    if so.dim() != 2 or so.shape[1] != 3:
        raise ValueError("seq_offsets must be [B+1, 3]")
    return so


class Index:
    """A libdosa handle: the certified indexer and its dense reference."""

    def __init__(self, dtype: str = "bf16", H: int = 64, d: int = 128, max_K: int = 2048,
                 **overrides):
        lib = load()
        cfg = Config()
        lib.dosa_index_config_default(ctypes.byref(cfg))
        cfg.H, cfg.d, cfg.max_K = H, d, max_K
        cfg.dtype = DOSA_FP8_E4M3 if dtype == "fp8" else DOSA_BF16
        for k, v in overrides.items():
            setattr(cfg, k, int(v))
        self.cfg = cfg
        self.dtype = dtype
        h = ctypes.c_void_p()
        _check("dosa_index_create", lib.dosa_index_create(ctypes.byref(cfg), ctypes.byref(h)))
        self._h = h
        self._lib = lib

    def close(self):
        if getattr(self, "_h", None):
            self._lib.dosa_index_destroy(self._h)
            self._h = None

    __del__ = close

    def workspace_size(self, Tq: int, S_max: int, K: int, certified: bool,
                       chunk_rows: int = 0) -> int:
        n = ctypes.c_size_t()
        _check("dosa_index_workspace_size",
               self._lib.dosa_index_workspace_size(self._h, Tq, S_max, K, int(certified),
                                                   chunk_rows, ctypes.byref(n)))
        return int(n.value)

    def _workspace(self, q, seq_offsets, K, certified, workspace):
        if workspace is not None:
            return workspace
        so = _seq_offsets(seq_offsets)
        S_max = int((so[1:, 1] - so[:-1, 1]).max())
        n = self.workspace_size(q.shape[0], S_max, K, certified)
        return torch.zeros(n, dtype=torch.uint8, device=q.device)

    def _topk_args(self, q, q_scale, w, k, k_scale, seq_offsets, K, out):
        so = _seq_offsets(seq_offsets)
        if out is None:
            out = torch.empty((q.shape[0], K), dtype=torch.int32, device=q.device)
        return so, out

    def dense_topk(self, q, q_scale, w, k, k_scale, seq_offsets, K, out=None, workspace=None):
        so, out = self._topk_args(q, q_scale, w, k, k_scale, seq_offsets, K, out)
        ws = self._workspace(q, so, K, False, workspace)
        _check("dosa_index_dense_topk", self._lib.dosa_index_dense_topk(
            self._h, _ptr(q), _ptr(q_scale), _ptr(w), _ptr(k), _ptr(k_scale),
            ctypes.c_void_p(so.data_ptr()), so.shape[0] - 1, K, _ptr(out), _ptr(ws),
            ws.numel(), _stream()))
        return out

    def topk(self, q, q_scale, w, k, k_scale, seq_offsets, K, out=None, workspace=None,
             stats: bool = False):
        so, out = self._topk_args(q, q_scale, w, k, k_scale, seq_offsets, K, out)
        ws = self._workspace(q, so, K, True, workspace)
        st = Stats()
        _check("dosa_index_topk", self._lib.dosa_index_topk(
            self._h, _ptr(q), _ptr(q_scale), _ptr(w), _ptr(k), _ptr(k_scale),
            ctypes.c_void_p(so.data_ptr()), so.shape[0] - 1, K, _ptr(out), _ptr(ws),
            ws.numel(), _stream(), ctypes.byref(st) if stats else None))
        return (out, st.as_dict()) if stats else out

    def host_workspace_size(self, Tq: int, S_total: int, S_max: int, K: int,
                            chunk_rows: int = 0) -> int:
        n = ctypes.c_size_t()
        _check("dosa_index_host_workspace_size",
               self._lib.dosa_index_host_workspace_size(self._h, Tq, S_total, S_max, K,
                                                        chunk_rows, ctypes.byref(n)))
        return int(n.value)

    def topk_host(self, q, q_scale, w, k, k_scale, seq_offsets, K, out=None, workspace=None,
                  stats: bool = False):
        """Certified Top-K with host (CPU, ideally pinned) inputs and output; the
        workspace is a CUDA tensor (host_workspace_size bytes)."""
        so = _seq_offsets(seq_offsets)
        if out is None:
            out = torch.empty((q.shape[0], K), dtype=torch.int32, pin_memory=True)
        if workspace is None:
            S_max = int((so[1:, 1] - so[:-1, 1]).max())
            n = self.host_workspace_size(q.shape[0], int(so[-1, 1]), S_max, K)
            workspace = torch.zeros(n, dtype=torch.uint8, device="cuda")
        st = Stats()
        _check("dosa_index_topk_host", self._lib.dosa_index_topk_host(
            self._h, _ptr(q), _ptr(q_scale), _ptr(w), _ptr(k), _ptr(k_scale),
            ctypes.c_void_p(so.data_ptr()), so.shape[0] - 1, K, _ptr(out), _ptr(workspace),
            workspace.numel(), _stream(), ctypes.byref(st) if stats else None))
        return (out, st.as_dict()) if stats else out

    def decode_workspace_size(self, Tq: int, S_max: int, K: int) -> int:
        n = ctypes.c_size_t()
        _check("dosa_index_decode_workspace_size",
               self._lib.dosa_index_decode_workspace_size(self._h, Tq, S_max, K, ctypes.byref(n)))
        return int(n.value)

    def decode_topk(self, q, q_scale, w, k, k_scale, seq_offsets, K, seed_idx, out=None,
                    workspace=None, stats: bool = False):
        """Decode-step Top-K seeded by the previous step's selection seed_idx [Tq, K]."""
        so, out = self._topk_args(q, q_scale, w, k, k_scale, seq_offsets, K, out)
        if workspace is None:
            S_max = int((so[1:, 1] - so[:-1, 1]).max())
            workspace = torch.zeros(self.decode_workspace_size(q.shape[0], S_max, K),
                                    dtype=torch.uint8, device=q.device)
        seed = seed_idx.to(torch.int32).contiguous()
        st = Stats()
        _check("dosa_index_decode_topk", self._lib.dosa_index_decode_topk(
            self._h, _ptr(q), _ptr(q_scale), _ptr(w), _ptr(k), _ptr(k_scale),
            ctypes.c_void_p(so.data_ptr()), so.shape[0] - 1, K, _ptr(seed), _ptr(out),
            _ptr(workspace), workspace.numel(), _stream(), ctypes.byref(st) if stats else None))
        return (out, st.as_dict()) if stats else out

    def certificate(self, q, q_scale, w, k, k_scale, seq_offsets, workspace=None,
                    bound_rows: bool = False):
        """Per-query certificate records [Tq, 16] (code domain), retained heads
        [Tq, 4] and, when asked, the bound rows [Tq, 8, d] (codes, q's dtype)."""
        so = _seq_offsets(seq_offsets)
        cert = torch.empty((q.shape[0], 16), dtype=torch.float32, device=q.device)
        ret = torch.empty((q.shape[0], 4), dtype=torch.int32, device=q.device)
        rows = (torch.empty((q.shape[0], 8, q.shape[2]), dtype=q.dtype, device=q.device)
                if bound_rows else None)
        ws = self._workspace(q, so, 1, True, workspace)
        _check("dosa_index_certificate", self._lib.dosa_index_certificate(
            self._h, _ptr(q), _ptr(q_scale), _ptr(w), _ptr(k), _ptr(k_scale),
            ctypes.c_void_p(so.data_ptr()), so.shape[0] - 1, _ptr(cert), _ptr(ret), _ptr(rows),
            _ptr(ws), ws.numel(), _stream()))
        return (cert, ret, rows) if bound_rows else (cert, ret)

    def scores(self, q, q_scale, w, k, k_scale, row0, rows, pos0, S, out, ld, scratch):
        _check("dosa_index_scores", self._lib.dosa_index_scores(
            self._h, _ptr(q), _ptr(q_scale), _ptr(w), _ptr(k), _ptr(k_scale), row0, rows, pos0,
            S, _ptr(out), ld, _ptr(scratch), _stream()))
        return out

    def reference_scores(self, q, q_scale, w, k, k_scale, row0, rows, pos0, S, out, ld):
        _check("dosa_reference_scores", self._lib.dosa_reference_scores(
            self._h, _ptr(q), _ptr(q_scale), _ptr(w), _ptr(k), _ptr(k_scale), row0, rows, pos0,
            S, _ptr(out), ld, _stream()))
        return out


ATTN_DTYPES = {"bf16": (DOSA_BF16, torch.bfloat16), "fp16": (DOSA_FP16, torch.float16)}


def _on_current_device(**tensors):
    """The kernels run on the current device's current stream: every tensor
    has to live there."""
    dev = torch.cuda.current_device()
    for name, t in tensors.items():
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name} must be on the current CUDA device (cuda:{dev}), "
                             f"not {t.device}")
    return dev


def _own_bytes(workspace, dev):
    """The kernels take a caller's workspace as one run of bytes on their device."""
    if workspace.get_device() != dev:
        _on_current_device(workspace=workspace)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")


_Pair = ctypes.c_int64 * 2


def _batch(seq_offsets):
    """(tensor, its address, B, rows, keys) of seq_offsets as the calls take them.
    The caller keeps the tensor until its call is made."""
    so = seq_offsets
    if not (type(so) is torch.Tensor and so.dtype is torch.int64 and so.dim() == 2 and
            so.size(1) == 3 and not so.is_cuda and so.is_contiguous()):
        so = _seq_offsets(so)
    B, at = so.size(0) - 1, so.data_ptr()
    if B < 1:
        raise ValueError("seq_offsets must be [B+1, 3] with B >= 1")
    Tq, S = _Pair.from_address(at + 24 * B)
    return so, at, B, Tq, S


class Cache4:
    """The 4-bit key/value cache (layout in include/dosa.h): codes uint8
    [Hkv, capacity, 64], params float16 [Hkv, capacity, 4, 2], weight float32
    [capacity] (None: attention weights are not recorded)."""

    def __init__(self, k_codes, k_params, v_codes, v_params, weight=None):
        Hkv, cap = k_codes.shape[0], k_codes.shape[1]
        for name, t, shape, dtype in (
                ("k_codes", k_codes, (Hkv, cap, 64), torch.uint8),
                ("v_codes", v_codes, (Hkv, cap, 64), torch.uint8),
                ("k_params", k_params, (Hkv, cap, 4, 2), torch.float16),
                ("v_params", v_params, (Hkv, cap, 4, 2), torch.float16),
                ("weight", weight, (cap,), torch.float32)):
            if t is None and name == "weight":
                continue
            if tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape}")
        self.k_codes, self.k_params = k_codes, k_params
        self.v_codes, self.v_params = v_codes, v_params
        self.weight = weight
        self.Hkv, self.capacity = Hkv, cap

    @classmethod
    def empty(cls, Hkv: int, capacity: int, weight: bool = True, device="cuda"):
        """A cache of zeroed slots."""
        z = lambda shape, dtype: torch.zeros(shape, dtype=dtype, device=device)
        codes, params = (Hkv, capacity, 64), (Hkv, capacity, 4, 2)
        return cls(z(codes, torch.uint8), z(params, torch.float16), z(codes, torch.uint8),
                   z(params, torch.float16), z((capacity,), torch.float32) if weight else None)

    def _arrays(self, dev) -> Cache4Arrays:
        kc, kp, vc, vp, w = self.k_codes, self.k_params, self.v_codes, self.v_params, self.weight
        if not (kc.get_device() == kp.get_device() == vc.get_device() == vp.get_device() == dev and
                (w is None or w.get_device() == dev)):
            _on_current_device(k_codes=kc, k_params=kp, v_codes=vc, v_params=vp, weight=w)
        return Cache4Arrays(kc.data_ptr(), kp.data_ptr(), vc.data_ptr(), vp.data_ptr(),
                            None if w is None else w.data_ptr(), self.capacity)


class Attention:
    """A libdosa handle: the layer's main attention beside the indexer.  Query
    heads Hq in groups of Hq / Hkv per key head; scale None = 1 / sqrt(d)."""

    def __init__(self, dtype: str = "bf16", Hq: int = 64, Hkv: int = 8, d: int = 128, scale=None):
        lib = load()
        if dtype not in ATTN_DTYPES:
            raise ValueError(f"dtype must be one of {sorted(ATTN_DTYPES)}")
        if scale is not None and not scale > 0:
            raise ValueError("scale must be positive")
        cfg = AttnConfig()
        lib.dosa_attn_config_default(ctypes.byref(cfg))
        cfg.Hq, cfg.Hkv, cfg.d = Hq, Hkv, d
        cfg.dtype = ATTN_DTYPES[dtype][0]
        cfg.scale = 0.0 if scale is None else scale
        h = ctypes.c_void_p()
        _check("dosa_attn_create", lib.dosa_attn_create(ctypes.byref(cfg), ctypes.byref(h)))
        self.cfg, self.dtype, self.torch_dtype = cfg, dtype, ATTN_DTYPES[dtype][1]
        self._h, self._lib = h, lib
        self._Hq, self._Hkv, self._d = cfg.Hq, cfg.Hkv, cfg.d     # plain ints

    def close(self):
        if getattr(self, "_h", None):
            self._lib.dosa_attn_destroy(self._h)
            self._h = None

    __del__ = close

    def _rows(self, name, t, heads, rows, dev=None) -> Rows:
        shape, d = t.shape, self._d
        if dev is not None and t.get_device() != dev:
            _on_current_device(**{name: t})
        if len(shape) != 3 or shape[1] != heads or shape[2] != d or shape[0] < rows:
            raise ValueError(f"{name} must be [{rows}, {heads}, {d}], not {tuple(shape)}")
        if t.dtype is not self.torch_dtype:
            raise ValueError(f"{name} must be {self.torch_dtype}, not {t.dtype}")
        rs, hs, es = t.stride()
        if es != 1:
            raise ValueError(f"{name}: the elements of a vector must be contiguous")
        # a stride of a dimension of size one is never used
        return Rows(t.data_ptr(), rs if shape[0] > 1 else heads * d, hs if heads > 1 else d)

    def prompt_workspace_size(self, seq_offsets) -> int:
        return self._prompt_ws(*_batch(seq_offsets)[:3])

    def _prompt_ws(self, so, at, B) -> int:
        n = ctypes.c_size_t()
        _check("dosa_attn_prompt_workspace_size", self._lib.dosa_attn_prompt_workspace_size(
            self._h, at, B, ctypes.byref(n)))
        return int(n.value)

    def _out(self, q, Tq, out, lse, dev):
        """(out, lse, its address)."""
        if out is None:
            out = q.new_empty((Tq, self._Hq, self._d))
        if lse is False or lse is None:
            return out, None, None
        if lse is True:
            lse = q.new_empty((Tq, self._Hq), dtype=torch.float32)
        elif (tuple(lse.shape) != (Tq, self._Hq) or lse.dtype != torch.float32 or
              not lse.is_contiguous()):
            raise ValueError(f"lse must be a contiguous float32 [{Tq}, {self._Hq}] tensor")
        if lse.get_device() != dev:
            _on_current_device(q=q, lse=lse)
        return out, lse, lse.data_ptr()

    def prompt(self, q, k, v, seq_offsets, out=None, lse=False, workspace=None):
        """Causal attention of packed rows q [Tq, Hq, d] over k, v [S, Hkv, d]
        (the indexer's seq_offsets).  lse: True (or a float32 [Tq, Hq] tensor)
        returns (out, lse)."""
        so, at, B, Tq, S = _batch(seq_offsets)
        dev, Hq, Hkv = torch.cuda.current_device(), self._Hq, self._Hkv
        qr = self._rows("q", q, Hq, Tq, dev)
        kr, vr = self._rows("k", k, Hkv, S, dev), self._rows("v", v, Hkv, S, dev)
        out, lse, lse_at = self._out(q, Tq, out, lse, dev)
        ws = workspace
        if ws is None:
            ws = q.new_zeros(self._prompt_ws(so, at, B), dtype=torch.uint8)
        else:
            _own_bytes(ws, dev)
        _check("dosa_attn_prompt", self._lib.dosa_attn_prompt(
            self._h, qr, kr, vr, at, B, self._rows("out", out, Hq, Tq, dev), lse_at,
            ws.data_ptr(), ws.nbytes, _stream(dev)))
        return out if lse is None else (out, lse)

    def append(self, cache: Cache4, k, v, seq_offsets):
        """Quantise the batch's rows k, v [Tq, Hkv, d] into their cache slots."""
        so, at, B, Tq, _ = _batch(seq_offsets)
        dev, Hkv = torch.cuda.current_device(), self._Hkv
        self._own_heads(cache)
        _check("dosa_cache4_append", self._lib.dosa_cache4_append(
            self._h, cache._arrays(dev), self._rows("k", k, Hkv, Tq, dev),
            self._rows("v", v, Hkv, Tq, dev), at, B, _stream(dev)))

    def read(self, cache: Cache4, seq_offsets, k=None, v=None):
        """The slots of the batch's rows as k, v [Tq, Hkv, d]."""
        so, at, B, Tq, _ = _batch(seq_offsets)
        dev, Hkv = torch.cuda.current_device(), self._Hkv
        self._own_heads(cache)
        arrays = cache._arrays(dev)
        if k is None:
            k = cache.k_codes.new_empty((Tq, Hkv, self._d), dtype=self.torch_dtype)
        if v is None:
            v = cache.k_codes.new_empty((Tq, Hkv, self._d), dtype=self.torch_dtype)
        _check("dosa_cache4_read", self._lib.dosa_cache4_read(
            self._h, arrays, at, B, self._rows("k", k, Hkv, Tq, dev),
            self._rows("v", v, Hkv, Tq, dev), _stream(dev)))
        return k, v

    def _own_heads(self, cache):
        if cache.Hkv != self._Hkv:
            raise ValueError(f"the cache has {cache.Hkv} key heads, the handle {self._Hkv}")

    def attend_workspace_size(self, seq_offsets, K: int = 0, weights: bool = False) -> int:
        return self._attend_ws(*_batch(seq_offsets)[:3], K, weights)

    def _attend_ws(self, so, at, B, K, weights) -> int:
        n = ctypes.c_size_t()
        _check("dosa_cache4_attend_workspace_size", self._lib.dosa_cache4_attend_workspace_size(
            self._h, at, B, K, int(weights), ctypes.byref(n)))
        return int(n.value)

    def attend(self, cache: Cache4, q, seq_offsets, sel_idx=None, weights: bool = False, out=None,
               lse=False, workspace=None):
        """Attention of rows q [Tq, Hq, d] over the cache: every visible key, or
        the keys sel_idx [Tq, K] lists (a Top-K call's result).  weights: add
        the attention weight each token received to cache.weight."""
        so, at, B, Tq, _ = _batch(seq_offsets)
        dev, Hq = torch.cuda.current_device(), self._Hq
        self._own_heads(cache)
        arrays = cache._arrays(dev)
        qr = self._rows("q", q, Hq, Tq, dev)
        out, lse, lse_at = self._out(q, Tq, out, lse, dev)
        K, sel_at = 0, None
        if sel_idx is not None:
            if (sel_idx.dim() != 2 or sel_idx.shape[0] != Tq or sel_idx.dtype != torch.int32 or
                    not sel_idx.is_contiguous()):
                raise ValueError(f"sel_idx must be a contiguous int32 [{Tq}, K] tensor")
            if sel_idx.get_device() != dev:
                _on_current_device(sel_idx=sel_idx)
            K, sel_at = sel_idx.shape[1], sel_idx.data_ptr()
            if K == 0:      # no list at all would mean every key
                raise ValueError("sel_idx must list at least one entry per row")
            if Tq == 0:
                K, sel_at = 0, None
        ws = workspace
        if ws is None:
            ws = q.new_zeros(self._attend_ws(so, at, B, K, weights), dtype=torch.uint8)
        else:
            _own_bytes(ws, dev)
        _check("dosa_cache4_attend", self._lib.dosa_cache4_attend(
            self._h, arrays, qr, at, B, sel_at, K, 1 if weights else 0,
            self._rows("out", out, Hq, Tq, dev), lse_at, ws.data_ptr(), ws.nbytes, _stream(dev)))
        return out if lse is None else (out, lse)

    def evict(self, src: Cache4, dst: Cache4, spans, first: int = 0, last: int = 0, kept=None):
        """Move each sequence's tokens that matter from src to dst.  spans (host)
        [B, 4] = src_start, n, dst_start, keep; returns kept [B, max keep] int32."""
        sp = spans
        if not (type(sp) is torch.Tensor and sp.dtype is torch.int64 and not sp.is_cuda and
                sp.is_contiguous()):
            sp = torch.as_tensor(spans, dtype=torch.int64).cpu().contiguous()
        if sp.dim() != 2 or sp.shape[1] != 4 or sp.shape[0] < 1:
            raise ValueError("spans must be [B, 4]")
        B, at, dev = sp.shape[0], sp.data_ptr(), torch.cuda.current_device()
        keep = max((ctypes.c_int64 * (4 * B)).from_address(at)[3::4])
        self._own_heads(src)
        self._own_heads(dst)
        sa, da = src._arrays(dev), dst._arrays(dev)
        if kept is None:
            kept = src.k_codes.new_empty((B, max(0, keep)), dtype=torch.int32)
        elif (kept.dim() != 2 or kept.shape[0] != B or kept.dtype != torch.int32 or
              not kept.is_contiguous()):
            raise ValueError(f"kept must be a contiguous int32 [{B}, keep] tensor")
        if kept.get_device() != dev:
            _on_current_device(kept=kept)
        _check("dosa_cache4_evict", self._lib.dosa_cache4_evict(
            self._h, sa, da, at, B, first, last, kept.data_ptr(), kept.shape[1], _stream(dev)))
        return kept


def topk_rows(scores: torch.Tensor, row_len: torch.Tensor, K: int, out=None) -> torch.Tensor:
    lib = load()
    if out is None:
        out = torch.empty((scores.shape[0], K), dtype=torch.int32, device=scores.device)
    _check("dosa_topk_rows", lib.dosa_topk_rows(_ptr(scores), scores.stride(0), _ptr(row_len),
                                                scores.shape[0], K, _ptr(out), _stream()))
    return out


def check_device(workspace: torch.Tensor):
    _check("dosa_check_device", load().dosa_check_device(_ptr(workspace), _stream()))


def profile_enable(on: bool = True):
    _check("dosa_profile_enable", load().dosa_profile_enable(int(on)))


def profile_reset():
    _check("dosa_profile_reset", load().dosa_profile_reset())


def profile_read() -> dict:
    """{kernel kind: (launches, summed device ms)} since the last reset."""
    lib = load()
    out = {}
    for name, kind in KERNELS.items():
        n, ms = ctypes.c_int64(), ctypes.c_double()
        _check("dosa_profile_read", lib.dosa_profile_read(kind, ctypes.byref(n), ctypes.byref(ms)))
        out[name] = (int(n.value), float(ms.value))
    return out

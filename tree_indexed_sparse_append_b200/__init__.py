"""Python binding of libzha, the B200 (sm_100a) library for Zyphra Hierarchical
Attention: a tree of compressed key summaries over a KV cache, walked top-down by
each query, followed by attention over exactly the keys the walk chose.

This module only marshals arguments (torch tensors -> device pointers, the current
CUDA stream) into the C ABI declared in include/zha.h; every step runs in the
library's CUDA kernels. There is no CPU fallback: without libzha.so or a CUDA
device the calls raise.

Names follow the C ABI: build / append / search / attend.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libzha.so")
MAX_DEPTH = 12

OK, ERR_INVALID, ERR_CAPACITY, ERR_OOM, ERR_CUDA, ERR_INTERNAL, ERR_TIMEOUT = 0, -1, -2, -3, -4, -5, -6
F32, BF16, E4M3 = 0, 1, 2
MAX_DRAFT = 1024
TOP_P, TOP_K = 0, 1

# Every symbol include/zha.h declares.
SYMBOLS = ("zha_build", "zha_append", "zha_search", "zha_attend", "zha_reserve", "zha_level",
           "zha_num_keys", "zha_depth", "zha_sync_status", "zha_destroy", "zha_last_error", "zha_version",
           "zha_profile", "zha_profile_read", "zha_kernel_launches", "zha_last_search_info",
           "zha_dense_scan", "zha_attend_noalloc", "zha_chunk_mass", "zha_ref_grad", "zha_rebuild",
           "zha_kv_write", "zha_kv_read", "zha_build_scaled", "zha_extend", "zha_attend_draft",
           "zha_test_wait_limit", "zha_cp_begin", "zha_cp_export", "zha_cp_select", "zha_lse_combine")
KERNEL_KINDS = ("build", "append", "search_init", "score", "select", "attend_plan", "attend_partial",
                "attend_combine", "score_tc")


class ZhaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"zha error {code}: {msg}")
        self.code = code


class Config(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("d", ctypes.c_int),
                ("R", ctypes.c_int), ("chunk", ctypes.c_int), ("depth", ctypes.c_int),
                ("top_width", ctypes.c_int), ("capacity", ctypes.c_longlong),
                ("sharpness", ctypes.c_float), ("kv_dtype", ctypes.c_int)]


class Stats(ctypes.Structure):
    _fields_ = [("start_level", ctypes.c_int), ("frontier", ctypes.c_int * (MAX_DEPTH + 1)),
                ("opened", ctypes.c_int * (MAX_DEPTH + 1)), ("keys_read", ctypes.c_longlong),
                ("work", ctypes.c_longlong)]


STATS_BYTES = ctypes.sizeof(Stats)


class KernelTime(ctypes.Structure):
    _fields_ = [("launches", ctypes.c_longlong), ("ms", ctypes.c_double)]


class SearchInfo(ctypes.Structure):
    _fields_ = [("start_level", ctypes.c_int), ("union_nodes", ctypes.c_longlong * (MAX_DEPTH + 1)),
                ("walk_nodes", ctypes.c_longlong * (MAX_DEPTH + 1))]

_lib = None


def lib():
    """The loaded libzha.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run __graft_entry__.build() (nvcc, sm_100a)")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, ll, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
        L.zha_build.argtypes = [ctypes.POINTER(Config), vp, vp, vp, ll, vp, ctypes.POINTER(vp)]
        L.zha_append.argtypes = [vp, vp, vp, vp]
        L.zha_kv_write.argtypes = [vp, vp, i, vp, vp, ll, i, i, i, vp, vp, vp, vp, ll, ll, vp]
        L.zha_kv_read.argtypes = [vp, vp, vp, vp, i, i, i, ll, ll, ll, vp, vp, i, vp]
        L.zha_build_scaled.argtypes = [ctypes.POINTER(Config), vp, vp, vp, vp, vp, ll, vp, ctypes.POINTER(vp)]
        L.zha_extend.argtypes = [vp, vp, vp, i, vp, vp, vp, ll, ll, vp]
        L.zha_attend_draft.argtypes = [vp, vp, i, i, i, vp, vp, i, vp, vp, i, vp, vp, i, vp, vp]
        L.zha_rebuild.argtypes = [vp, vp]
        L.zha_test_wait_limit.argtypes = [vp, ll, i]
        L.zha_cp_begin.argtypes = [vp, vp, i, i, i, ll, ctypes.POINTER(ll), i, ctypes.POINTER(i), vp]
        L.zha_cp_export.argtypes = [vp, vp, vp, vp, ll, ctypes.POINTER(i), vp]
        L.zha_cp_select.argtypes = [vp, i, vp, vp, vp, ll, i, f, i, vp, vp, i, ctypes.POINTER(i), vp]
        L.zha_lse_combine.argtypes = [i, ll, i, vp, vp, vp, i, vp, vp]
        L.zha_search.argtypes = [vp, vp, i, i, i, i, f, i, vp, vp, i, vp, vp]
        L.zha_attend.argtypes = [vp, vp, i, i, i, vp, vp, i, vp, i, vp, vp]
        L.zha_attend_noalloc.argtypes = [vp, vp, i, i, i, vp, vp, i, vp, i, vp, vp]
        L.zha_reserve.argtypes = [vp, ll, i]
        L.zha_dense_scan.argtypes = [vp, vp, i, i, i, i, f, i, vp, vp, i, vp]
        L.zha_chunk_mass.argtypes = [vp, vp, i, i, i, i, f, vp, vp, i, vp]
        L.zha_ref_grad.argtypes = [vp, vp, i, i, i, vp, vp, vp]
        L.zha_level.argtypes = [vp, i, ctypes.POINTER(vp), ctypes.POINTER(ll), ctypes.POINTER(ll),
                                ctypes.POINTER(i)]
        L.zha_num_keys.argtypes = [vp]
        L.zha_num_keys.restype = ll
        L.zha_depth.argtypes = [vp]
        L.zha_depth.restype = ctypes.c_int
        L.zha_sync_status.argtypes = [vp, vp]
        L.zha_destroy.argtypes = [vp]
        L.zha_destroy.restype = None
        L.zha_profile.argtypes = [vp, i]
        L.zha_profile_read.argtypes = [vp, ctypes.POINTER(KernelTime), vp]
        L.zha_kernel_launches.restype = ll
        L.zha_kernel_launches.argtypes = []
        L.zha_last_search_info.argtypes = [vp, ctypes.POINTER(SearchInfo), vp]
        L.zha_last_error.restype = ctypes.c_char_p
        L.zha_version.restype = ctypes.c_char_p
        for name in SYMBOLS:
            getattr(L, name)
        _lib = L
    return _lib


def _check(rc: int):
    if rc != OK:
        raise ZhaError(rc, lib().zha_last_error().decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t.dtype}: use float32 or bfloat16")


def _cache_code(t: torch.Tensor) -> int:
    return E4M3 if t.dtype == torch.float8_e4m3fn else _dtype_code(t)


_SCALE_DTYPES = (torch.uint8, getattr(torch, "float8_e8m0fnu", torch.uint8))


def _scale(t, K: torch.Tensor, dev: int, name: str) -> int:
    """Exponent bytes of an 8-bit cache K [B][H_kv][capacity][d]."""
    if t is None or t.dtype not in _SCALE_DTYPES or t.shape != K.shape[:3]:
        raise ValueError(f"{name} must be uint8 (or float8_e8m0fnu) [B][H_kv][capacity] for an E4M3 cache")
    return _dev_of(t, name, dev)


def _dev_of(t: torch.Tensor, name: str, dev: int) -> int:
    """t's pointer; t must be contiguous and on CUDA device dev."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev} (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _cuda_index(t: torch.Tensor, name: str) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


_Strides = ctypes.c_longlong * 3


def _rows(t: torch.Tensor, name: str, dev: int):
    """(pointer, element strides) of rows [B][H_kv][m][d] read in place: any strides
    but the last dimension's, which must be 1."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev} (got {t.device})")
    b, h, r, c = t.stride()
    if c != 1 and t.shape[3] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    if 1 in t.shape:  # the stride of a dimension of one element means nothing
        B, H, m, _ = t.shape
        b, h, r = (0 if B == 1 else b), (0 if H == 1 else h), (0 if m == 1 else r)
    return t.data_ptr(), _Strides(b, h, r)


def _launch(f, dev: int, stream, *args) -> None:
    """Calls f(*args, stream) with the tensors' device current (a tree's own, whichever was),
    on its current stream unless one is given."""
    s = stream.cuda_stream if stream is not None else _raw_stream(dev)
    if _get_device() == dev:
        rc = f(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = f(*args, s)
    if rc != OK:
        _check(rc)


# the current stream's handle and the current device, without the objects around
# them (torch.cuda.current_stream() takes 3 us) where torch has these names: one
# built without CUDA lacks them
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_get_device = getattr(torch._C, "_cuda_getDevice", None) or (lambda: torch.cuda.current_device())


class _DeviceArray:
    """A non-owning __cuda_array_interface__ view of library-owned device memory."""

    def __init__(self, ptr: int, shape, typestr: str, owner):
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr,
                                         "data": (ptr, False), "version": 3, "strides": None}
        self._owner = owner


class Tree:
    """The summary trees of a KV cache [B][H_kv][capacity][d] (one per sequence and
    KV head). K, V and refs stay referenced here: the library keeps their pointers.

    An 8-bit cache is float8_e4m3fn K and V with their exponent bytes, k_scale and
    v_scale [B][H_kv][capacity] (uint8 or float8_e8m0fnu): see kv_write."""

    def __init__(self, K: torch.Tensor, V: torch.Tensor, refs: torch.Tensor, n_keys: int, chunk: int,
                 depth: int, sharpness: float, top_width: int = 64, stream=None,
                 k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None):
        if K.dim() != 4 or V.shape != K.shape:
            raise ValueError("K and V must both be [B][H_kv][capacity][d]")
        if refs.dim() != 3 or refs.dtype != torch.float32 or refs.shape[0] != K.shape[1] or refs.shape[2] != K.shape[3]:
            raise ValueError("refs must be fp32 [H_kv][R][d]")
        if V.dtype != K.dtype:
            raise ValueError("K and V must have the same dtype")
        B, H, cap, d = K.shape
        self.cfg = Config(batch=B, n_kv_heads=H, d=d, R=refs.shape[1], chunk=chunk, depth=depth,
                          top_width=top_width, capacity=cap, sharpness=sharpness,
                          kv_dtype=_cache_code(K))
        self.K, self.V, self.refs = K, V, refs
        self.k_scale, self.v_scale = k_scale, v_scale
        self._h = ctypes.c_void_p()
        self._device = dev = _cuda_index(K, "K")
        if self.cfg.kv_dtype == E4M3:
            build = lib().zha_build_scaled
            scales = _scale(k_scale, K, dev, "k_scale"), _scale(v_scale, K, dev, "v_scale")
        else:
            build, scales = lib().zha_build, ()
            if k_scale is not None or v_scale is not None:
                raise ValueError("k_scale and v_scale belong to an E4M3 cache")
        _launch(lambda *a: build(*a, ctypes.byref(self._h)), dev, stream, ctypes.byref(self.cfg), _dev_of(K, "K", dev),
                _dev_of(V, "V", dev), *scales, _dev_of(refs, "refs", dev), int(n_keys))

    # -- properties -------------------------------------------------------
    @property
    def handle(self) -> int:
        return self._h.value

    @property
    def n_keys(self) -> int:
        return int(lib().zha_num_keys(self._h))

    @property
    def depth(self) -> int:
        """Levels the trees have now (the configured depth, or for depth=0 the
        deepest level holding a node)."""
        return int(lib().zha_depth(self._h))

    def level_sizes(self) -> list:
        out = [self.n_keys]
        for l in range(1, self.depth + 1):
            out.append(self.level(l)[1])
        return out

    def level(self, l: int):
        """(nodes view [B*H_kv][level_capacity][node_floats] fp32, live node count)."""
        ptr = ctypes.c_void_p()
        n = ctypes.c_longlong()
        cap = ctypes.c_longlong()
        nf = ctypes.c_int()
        _check(lib().zha_level(self._h, l, ctypes.byref(ptr), ctypes.byref(n), ctypes.byref(cap),
                               ctypes.byref(nf)))
        T = self.cfg.batch * self.cfg.n_kv_heads
        if not ptr.value:
            return torch.zeros(T, 0, nf.value, device=self.K.device), n.value
        view = torch.as_tensor(_DeviceArray(ptr.value, (T, cap.value, nf.value), "<f4", self),
                               device=self.K.device)
        return view, n.value

    # -- the hot path -----------------------------------------------------
    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> None:
        """One key and value [B][H_kv][d] per tree, of the cache dtype (for an E4M3
        cache: fp32 or bf16, quantised as they are written)."""
        B, H, _, d = self.K.shape
        if self.cfg.kv_dtype == E4M3:
            if k_new.shape != (B, H, d) or v_new.shape != (B, H, d):
                raise ValueError("k_new and v_new must be [B][H_kv][d]")
            return self.extend(k_new.unsqueeze(2), v_new.unsqueeze(2), stream=stream)
        if k_new.shape != (B, H, d) or v_new.shape != (B, H, d) or k_new.dtype != self.K.dtype or v_new.dtype != self.K.dtype:
            raise ValueError("k_new and v_new must be [B][H_kv][d] of the cache dtype")
        dev = self._device
        _launch(lib().zha_append, dev, stream, self._h, _dev_of(k_new, "k_new", dev), _dev_of(v_new, "v_new", dev))

    def extend(self, k_new: torch.Tensor, v_new: torch.Tensor, rows: torch.Tensor | None = None,
               stream=None) -> None:
        """Append m keys and values per tree, k_new and v_new [B][H_kv][m][d] (any
        strides with contiguous rows), and make the nodes they fill. An E4M3 cache
        takes fp32 or bf16 rows and quantises them as they are written; another cache
        takes rows of its dtype. With rows, int32 [B][m], key i of sequence b is
        k_new[b, :, rows[b, i]]: the accepted path of drafted tokens."""
        B, H, _, d = self.K.shape
        if k_new.dim() != 4 or k_new.shape[:2] != (B, H) or k_new.shape[3] != d or v_new.shape != k_new.shape:
            raise ValueError("k_new and v_new must both be [B][H_kv][m][d]")
        if v_new.dtype != k_new.dtype or (self.cfg.kv_dtype != E4M3 and k_new.dtype != self.K.dtype):
            raise ValueError("k_new and v_new must be of one dtype, the cache's unless it is E4M3")
        src_rows = m = k_new.shape[2]
        dev = self._device
        if rows is not None:
            if rows.dtype != torch.int32 or rows.dim() != 2 or rows.shape[0] != B:
                raise ValueError("rows must be int32 [B][m]")
            m = rows.shape[1]
        if m == 0:
            return
        (kp, ks), (vp, vs) = _rows(k_new, "k_new", dev), _rows(v_new, "v_new", dev)
        _launch(lib().zha_extend, dev, stream, self._h, kp, vp, _dtype_code(k_new), ks, vs,
                _dev_of(rows, "rows", dev) if rows is not None else None, src_rows, m)

    def read(self, start: int, count: int, dtype=torch.bfloat16, stream=None):
        """Keys start .. start + count - 1 of an E4M3 cache and their values, as the
        values they stand for: (k, v) [B][H_kv][count][d]."""
        if self.cfg.kv_dtype != E4M3:
            raise ValueError("read() reads an E4M3 cache back; another cache is K and V themselves")
        if start < 0 or count < 0 or start + count > self.n_keys:
            raise ValueError(f"keys {start} .. {start + count} are not among the tree's {self.n_keys}")
        return kv_read(self.K, self.V, self.k_scale, self.v_scale, start, count, dtype, stream=stream)

    def rebuild(self, stream=None) -> None:
        """Summarize every level again in place from the cache and the current
        refs (after the refs were updated in place); allocates nothing."""
        _launch(lib().zha_rebuild, self._device, stream, self._h)

    def search(self, Q: torch.Tensor, mode: int = TOP_P, p: float = 0.9, k: int = 1, max_sel: int | None = None,
               with_stats: bool = False, out=None, stream=None):
        """Q: [B][H_q][n_q][d]. Returns (sel [walks][max_sel] int32, sel_count [walks] int32,
        stats uint8 [walks][sizeof zha_stats] or None)."""
        B, Hq, nq, d = Q.shape
        W = B * Hq * nq
        if max_sel is None:
            max_sel = max(1, self.level(1)[1])
        if out is None:
            sel = torch.empty(W, max_sel, dtype=torch.int32, device=Q.device)
            cnt = torch.empty(W, dtype=torch.int32, device=Q.device)
            st = torch.empty(W, STATS_BYTES, dtype=torch.uint8, device=Q.device) if with_stats else None
        else:
            sel, cnt, st = out
        dev = self._device
        _launch(lib().zha_search, dev, stream, self._h, _dev_of(Q, "Q", dev), _dtype_code(Q), Hq, nq, mode, float(p),
                int(k), _dev_of(sel, "sel", dev), _dev_of(cnt, "sel_count", dev), max_sel,
                _dev_of(st, "stats", dev) if st is not None else None)
        return sel, cnt, st

    def attend(self, Q: torch.Tensor, sel: torch.Tensor, sel_count: torch.Tensor, out=None, lse=None,
               out_dtype=None, stream=None):
        """Attention of each walk over its chosen chunks (distinct ids, in any order) and
        the tail. Returns (out [B][H_q][n_q][d] of out_dtype (default: the cache dtype; of
        an E4M3 cache, Q's), lse [walks] fp32)."""
        B, Hq, nq, d = Q.shape
        W = B * Hq * nq
        if out is None:
            out = torch.empty_like(Q, dtype=out_dtype or self._out_dtype(Q), memory_format=torch.contiguous_format)
        if lse is None:
            lse = Q.new_empty(W, dtype=torch.float32)
        dev = self._device
        _launch(lib().zha_attend, dev, stream, self._h, _dev_of(Q, "Q", dev), _dtype_code(Q), Hq, nq,
                _dev_of(sel, "sel", dev), _dev_of(sel_count, "sel_count", dev), sel.shape[1], _dev_of(out, "out", dev),
                _dtype_code(out), _dev_of(lse, "lse", dev))
        return out, lse

    def _out_dtype(self, Q: torch.Tensor):
        return Q.dtype if self.cfg.kv_dtype == E4M3 else self.K.dtype

    def attend_draft(self, Q: torch.Tensor, sel: torch.Tensor, sel_count: torch.Tensor, k_draft: torch.Tensor,
                     v_draft: torch.Tensor, mask: torch.Tensor, out=None, lse=None, out_dtype=None, stream=None):
        """Attention of n drafted tokens per sequence, Q [B][H_q][n][d]: each over its
        walk's chosen keys and the tail, as attend(), and over the drafted tokens
        that its row of mask [B][n][n] (bool or uint8) names. k_draft, v_draft
        [B][H_kv][n][d], fp32 or bf16. Returns (out, lse) as attend()."""
        B, H, _, d = self.K.shape
        dev = self._device
        if Q.dim() != 4 or Q.shape[0] != B or Q.shape[3] != d or Q.shape[1] % H:
            raise ValueError("Q must be [B][H_q][n][d], H_q a multiple of H_kv")
        Hq, n = Q.shape[1], Q.shape[2]
        W = B * Hq * n
        if k_draft.shape != (B, H, n, d) or v_draft.shape != k_draft.shape or v_draft.dtype != k_draft.dtype:
            raise ValueError("k_draft and v_draft must both be [B][H_kv][n][d], of one dtype")
        if mask.shape != (B, n, n) or mask.dtype not in (torch.bool, torch.uint8):
            raise ValueError("mask must be bool or uint8 [B][n][n]")
        if sel.dtype != torch.int32 or sel.dim() != 2 or sel.shape[0] != W or \
                sel_count.dtype != torch.int32 or sel_count.shape != (W,):
            raise ValueError("sel must be int32 [walks][max_sel] and sel_count int32 [walks]")
        q = _dev_of(Q, "Q", dev)
        if out is None:
            out = torch.empty_like(Q, dtype=out_dtype or self._out_dtype(Q))
        elif out.shape != Q.shape:
            raise ValueError("out must be [B][H_q][n][d]")
        if lse is None:
            lse = Q.new_empty(W, dtype=torch.float32)
        elif lse.dtype != torch.float32 or lse.numel() != W:
            raise ValueError("lse must be fp32 [walks]")
        _launch(lib().zha_attend_draft, dev, stream, self._h, q, _dtype_code(Q), Hq, n, _dev_of(sel, "sel", dev),
                _dev_of(sel_count, "sel_count", dev), sel.shape[1], _dev_of(k_draft, "k_draft", dev),
                _dev_of(v_draft, "v_draft", dev), _dtype_code(k_draft), _dev_of(mask, "mask", dev),
                _dev_of(out, "out", dev), _dtype_code(out), _dev_of(lse, "lse", dev))
        return out, lse

    def attend_noalloc(self, Q: torch.Tensor, sel: torch.Tensor, sel_count: torch.Tensor, out: torch.Tensor,
                       lse: torch.Tensor | None = None, stream=None):
        """attend() for callers whose device memory may not be allocated by the library:
        zha_attend_noalloc uses a fixed static device array as scratch. The caller
        provides out (and lse) already allocated; nothing is allocated here."""
        B, Hq, nq, d = Q.shape
        dev = self._device
        _launch(lib().zha_attend_noalloc, dev, stream, self._h, _dev_of(Q, "Q", dev), _dtype_code(Q), Hq, nq,
                _dev_of(sel, "sel", dev), _dev_of(sel_count, "sel_count", dev), sel.shape[1], _dev_of(out, "out", dev),
                _dtype_code(out), _dev_of(lse, "lse", dev) if lse is not None else None)
        return out, lse

    def dense_scan(self, Q: torch.Tensor, mode: int = TOP_P, p: float = 0.9, k: int = 1,
                   max_sel: int | None = None, out=None, stream=None):
        """Full-scan indexer: every key scored, top-p / top-K over keys.
        Returns (sel [walks][max_sel] int32 key indices ascending, sel_count [walks])."""
        B, Hq, nq, d = Q.shape
        W = B * Hq * nq
        if max_sel is None:
            max_sel = max(1, self.n_keys)
        if out is None:
            sel = torch.empty(W, max_sel, dtype=torch.int32, device=Q.device)
            cnt = torch.empty(W, dtype=torch.int32, device=Q.device)
        else:
            sel, cnt = out
        dev = self._device
        _launch(lib().zha_dense_scan, dev, stream, self._h, _dev_of(Q, "Q", dev), _dtype_code(Q), Hq, nq, mode,
                float(p), int(k), _dev_of(sel, "sel", dev), _dev_of(cnt, "sel_count", dev), max_sel)
        return sel, cnt

    def chunk_mass(self, Q: torch.Tensor, group: int = 16, p: float = 0.9, max_sel: int | None = None, out=None,
                   stream=None):
        """Chunk-mass profile of dense attention: per walk, the fewest chunks of
        `group` keys holding p of the softmax over all keys. Returns (sel
        [walks][max_sel] int32 chunk indices ascending, count [walks] int32,
        n_chunks)."""
        B, Hq, nq, d = Q.shape
        W = B * Hq * nq
        n_chunks = (self.n_keys + group - 1) // group if group >= 1 else 0
        if max_sel is None:
            max_sel = max(1, n_chunks)
        if out is None:
            sel = torch.empty(W, max_sel, dtype=torch.int32, device=Q.device)
            cnt = torch.empty(W, dtype=torch.int32, device=Q.device)
        else:
            sel, cnt = out
        dev = self._device
        _launch(lib().zha_chunk_mass, dev, stream, self._h, _dev_of(Q, "Q", dev), _dtype_code(Q), Hq, nq, int(group),
                float(p), _dev_of(sel, "sel", dev), _dev_of(cnt, "count", dev), max_sel)
        return sel, cnt, n_chunks

    def ref_grad(self, Q: torch.Tensor, stream=None):
        """The split loss (KL of the teacher's split of attention from the tree's,
        summed over levels, averaged over walks) and its gradient with respect to
        the references the tree was built with. Returns (loss [1], grad
        [H_kv][R][d]), fp32 on the device."""
        B, Hq, nq, d = Q.shape
        loss = torch.empty(1, dtype=torch.float32, device=Q.device)
        grad = torch.empty(self.cfg.n_kv_heads, self.cfg.R, d, dtype=torch.float32, device=Q.device)
        dev = self._device
        _launch(lib().zha_ref_grad, dev, stream, self._h, _dev_of(Q, "Q", dev), _dtype_code(Q), Hq, nq,
                _dev_of(loss, "loss", dev), _dev_of(grad, "grad", dev))
        return loss, grad

    # -- context-parallel walk (one shard of every tree per process) ------------
    def cp_begin(self, Q: torch.Tensor, key_begin: int, global_counts, stream=None) -> int:
        """Start a context-parallel walk of Q on this shard; returns the start level."""
        B, Hq, nq, d = Q.shape
        counts = (ctypes.c_longlong * len(global_counts))(*[int(c) for c in global_counts])
        level = ctypes.c_int()
        dev = self._device
        _launch(lib().zha_cp_begin, dev, stream, self._h, _dev_of(Q, "Q", dev), _dtype_code(Q), Hq, nq, int(key_begin),
                counts, len(global_counts), ctypes.byref(level))
        return level.value

    def cp_export(self, ids: torch.Tensor, scores: torch.Tensor, counts: torch.Tensor, stream=None) -> int:
        """Score this shard's frontier; ids/scores [walks][stride], counts [walks]. Returns the level."""
        level = ctypes.c_int()
        dev = self._device
        _launch(lib().zha_cp_export, dev, stream, self._h, _dev_of(ids, "ids", dev), _dev_of(scores, "scores", dev),
                _dev_of(counts, "counts", dev), ids.shape[1], ctypes.byref(level))
        return level.value

    def cp_select(self, ids: torch.Tensor, scores: torch.Tensor, counts: torch.Tensor, mode: int, p: float, k: int,
                  sel: torch.Tensor, sel_count: torch.Tensor, stream=None) -> int:
        """Choose over the gathered lists (ids/scores [parts][walks][stride], counts
        [parts][walks]); returns the next level (0 when the walk is complete)."""
        level = ctypes.c_int()
        dev = self._device
        _launch(lib().zha_cp_select, dev, stream, self._h, ids.shape[0], _dev_of(ids, "ids", dev),
                _dev_of(scores, "scores", dev), _dev_of(counts, "counts", dev), ids.shape[2], mode, float(p), int(k),
                _dev_of(sel, "sel", dev), _dev_of(sel_count, "sel_count", dev), sel.shape[1], ctypes.byref(level))
        return level.value

    def reserve(self, max_walks: int, max_sel: int) -> None:
        with torch.cuda.device(self._device):
            _check(lib().zha_reserve(self._h, int(max_walks), int(max_sel)))

    # -- diagnostics --------------------------------------------------------
    def profile(self, enable: bool) -> None:
        _check(lib().zha_profile(self._h, 1 if enable else 0))

    def profile_read(self, stream=None) -> dict:
        arr = (KernelTime * len(KERNEL_KINDS))()
        _launch(lib().zha_profile_read, self._device, stream, self._h, arr)
        return {name: (arr[i].launches, arr[i].ms) for i, name in enumerate(KERNEL_KINDS)}

    def last_search_info(self, stream=None) -> dict:
        info = SearchInfo()
        _launch(lib().zha_last_search_info, self._device, stream, self._h, ctypes.byref(info))
        return {"start_level": info.start_level, "union_nodes": list(info.union_nodes),
                "walk_nodes": list(info.walk_nodes)}

    def test_wait_limit(self, wait_ns: int, stall: bool = False) -> None:
        """Test hook: the tensor-core scorer's waits give up after wait_ns (0: the
        default 1 s); with stall, its launches first wait on a barrier nothing
        arrives at, so the search reports ZHA_ERR_TIMEOUT."""
        _check(lib().zha_test_wait_limit(self._h, int(wait_ns), 1 if stall else 0))

    def sync_status(self, stream=None) -> None:
        _launch(lib().zha_sync_status, self._device, stream, self._h)

    def close(self) -> None:
        if self._h and self._h.value:
            lib().zha_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def kv_write(k: torch.Tensor, v: torch.Tensor, K: torch.Tensor, V: torch.Tensor, k_scale: torch.Tensor,
             v_scale: torch.Tensor, start: int, stream=None) -> None:
    """Quantise k and v [B][H_kv][m][d] (fp32 or bf16, any strides with contiguous
    rows) into rows start .. start + m - 1 of an 8-bit cache: K, V [B][H_kv][capacity][d]
    float8_e4m3fn and their exponent bytes k_scale, v_scale [B][H_kv][capacity]
    (uint8 or float8_e8m0fnu). A row stands for code * 2^(byte - 127); the power is
    the least with max|x| <= 448 * 2^power (held in -117 .. 119)."""
    B, H, cap, d = _check_cache8(K, V)
    dev = _cuda_index(K, "K")
    if k.dim() != 4 or k.shape[:2] != (B, H) or k.shape[3] != d or v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("k and v must both be [B][H_kv][m][d], of one dtype")
    m = k.shape[2]
    if m == 0 and 0 <= start <= cap:
        return
    (kp, ks), (vp, vs) = _rows(k, "k", dev), _rows(v, "v", dev)
    _launch(lib().zha_kv_write, dev, stream, kp, vp, _dtype_code(k), ks, vs, m, B, H, d, _dev_of(K, "K", dev),
            _dev_of(V, "V", dev), _scale(k_scale, K, dev, "k_scale"), _scale(v_scale, K, dev, "v_scale"), cap,
            int(start))


def kv_read(K: torch.Tensor, V: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor, start: int, count: int,
            dtype=torch.bfloat16, stream=None):
    """Rows start .. start + count - 1 of an 8-bit cache as the values they stand for:
    (k, v) [B][H_kv][count][d] of dtype (bf16 or fp32; exact in both)."""
    B, H, cap, d = _check_cache8(K, V)
    dev = _cuda_index(K, "K")
    if count < 0:
        raise ValueError("count must be >= 0")
    if start < 0 or start + count > cap:
        raise ValueError(f"rows {start} .. {start + count} are not in a cache of {cap}")
    k = K.new_empty((B, H, count, d), dtype=dtype)
    v = torch.empty_like(k)
    _launch(lib().zha_kv_read, dev, stream, _dev_of(K, "K", dev), _dev_of(V, "V", dev),
            _scale(k_scale, K, dev, "k_scale"), _scale(v_scale, K, dev, "v_scale"), B, H, d, cap, int(start),
            int(count), k.data_ptr(), v.data_ptr(), _dtype_code(k))
    return k, v


def _check_cache8(K: torch.Tensor, V: torch.Tensor):
    if K.dtype != torch.float8_e4m3fn or V.dtype != K.dtype or K.dim() != 4 or V.shape != K.shape:
        raise ValueError("K and V must both be float8_e4m3fn [B][H_kv][capacity][d]")
    return K.shape


def lse_combine(outs: torch.Tensor, lses: torch.Tensor, out_dtype=torch.float32, stream=None):
    """Attention over the union of disjoint key sets: outs [parts][walks][d] fp32,
    lses [parts][walks] fp32 -> (out [walks][d] of out_dtype, lse [walks])."""
    P, W, d = outs.shape
    dev = _cuda_index(outs, "outs")
    out = torch.empty(W, d, dtype=out_dtype, device=outs.device)
    lse = torch.empty(W, dtype=torch.float32, device=outs.device)
    _launch(lib().zha_lse_combine, dev, stream, P, W, d, _dev_of(outs, "outs", dev), _dev_of(lses, "lses", dev),
            _dev_of(out, "out", dev), _dtype_code(out), _dev_of(lse, "lse", dev))
    return out, lse


def parse_stats(st: torch.Tensor) -> list:
    """Device stats bytes -> list of dicts (host)."""
    raw = st.cpu().numpy().tobytes()
    out = []
    for w in range(st.shape[0]):
        s = Stats.from_buffer_copy(raw[w * STATS_BYTES:(w + 1) * STATS_BYTES])
        out.append({"start_level": s.start_level, "frontier": list(s.frontier), "opened": list(s.opened),
                    "keys_read": s.keys_read, "work": s.work})
    return out


def kernel_launches() -> int:
    """Kernels this library has launched in this process."""
    return int(lib().zha_kernel_launches())


def version() -> str:
    return lib().zha_version().decode()

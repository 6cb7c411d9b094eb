"""Python binding of libbsa — 3D block-sparse attention for video DiTs on B200.

Argument marshalling only: every step runs in the CUDA kernels of
``libbsa.so`` (built in-tree by ``python -m block_sparse_attention_permute_b200.build``).
There is no fallback: importing works without the library, but every call
raises ``BsaError`` if ``libbsa.so`` is missing or the tensors are not on a
CUDA device.  PyTorch provides device memory and streams.

The calls mirror include/bsa.h (SPADE §3.3 "Head-wise Sparse Attention"):
``Plan.permute``/``unpermute`` (blocked layout), ``Plan.select`` (centroid
scores and Top-K / Top-P), ``Plan.attention`` (flash block-sparse attention)
and ``Plan.forward`` (all four in sequence).
"""
from __future__ import annotations

import array
import ctypes
import os

import torch

__all__ = ["Plan", "Rope", "CrossAttention", "BsaError", "TOPK", "TOPP", "lib_path", "load"]

TOPK = 0
TOPP = 1
_DT = {torch.float32: 0, torch.bfloat16: 1}
_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libbsa.so")
_lib = None


class BsaError(RuntimeError):
    """A libbsa call returned an error status (or the library is unavailable)."""

    def __init__(self, status: int, msg: str):
        super().__init__(f"libbsa status {status}: {msg}")
        self.status = status


class PlanInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in
                ("batch", "T", "H", "W", "bf", "br", "bc", "heads", "head_dim", "n_text", "dtype",
                 "Tp", "Hp", "Wp", "nbt", "nby", "nbx", "nb", "nb_text", "bs")] + \
               [("n_video", ctypes.c_longlong), ("n_tot", ctypes.c_longlong),
                ("npad_tot", ctypes.c_longlong), ("attn_path", ctypes.c_int)]


def lib_path() -> str:
    return _LIB_PATH


def load():
    """Load libbsa.so (raises BsaError if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise BsaError(-1, f"{_LIB_PATH} is missing; build it with "
                           "`python -m block_sparse_attention_permute_b200.build`")
    L = ctypes.CDLL(_LIB_PATH)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.bsa_last_error_string.restype = ctypes.c_char_p
    L.bsa_version.restype = I
    sigs = {
        "bsa_plan_create": [ctypes.POINTER(P)] + [I] * 11,
        "bsa_plan_destroy": [P],
        "bsa_plan_get_info": [P, ctypes.POINTER(PlanInfo)],
        "bsa_kmax_for": [P, I, P, ctypes.POINTER(I)],
        "bsa_workspace_size": [P, I, ctypes.POINTER(Z), ctypes.POINTER(Z)],
        "bsa_permute": [P, P, P, P, P],
        "bsa_permute_qkv": [P] * 10,
        "bsa_unpermute": [P, P, P, P],
        "bsa_centroids": [P, P, P, P, P, P],
        "bsa_attention_orig": [P, P, P, P, P, P, I, P, P, P],
        "bsa_select": [P, P, P, I, P, I, P, P, P, P, Z, P],
        "bsa_select_centroids": [P, P, P, I, P, I, P, P, P, P],
        "bsa_attention": [P, P, P, P, P, P, I, P, P, P],
        "bsa_forward": [P, P, P, P, I, P, I, P, P, P, P, Z, P, P],
        "bsa_check_status": [P, P],
        "bsa_plan_set_watchdog": [P, ctypes.c_longlong, I],
        "bsa_forward_timed": [P, P, P, P, I, P, I, P, P, P, P, Z, P, P, ctypes.POINTER(Timings)],
        "bsa_sics": [P, P, P, P],
        "bsa_kmax_for_union": [P, I, P, P, ctypes.POINTER(I)],
        "bsa_union_workspace_size": [P, I, P, ctypes.POINTER(Z), ctypes.POINTER(Z)],
        "bsa_select_union": [P, P, P, I, P, P, P, I, P, P, P, P, Z, P],
        "bsa_forward_union": [P, P, P, P, I, P, P, I, P, P, P, P, Z, P, P],
        "bsa_box_summaries": [P, P, P, P, P, P],
        "bsa_select_box": [P, I, P, P, I, P, P, P, I, P, P, P, P, Z, P],
        "bsa_estimator_workspace_size": [P, I, I, P, ctypes.POINTER(Z)],
        "bsa_forward_estimator": [P, P, P, P, I, I, P, P, I, P, P, P, P, Z, P, P],
        "bsa_grouped_workspace_size": [P, I, P, P, ctypes.POINTER(Z)],
        "bsa_pair_workspace_size": [P, I, ctypes.POINTER(Z)],
        "bsa_pair_tiles": [P, P, P, I, P, Z, P],
        "bsa_attention_paired": [P, P, P, P, P, P, I, P, Z, P, P, P],
        "bsa_forward_grouped": [P, I, P, P, P, P, I, P, P, P, P, P, P, P, Z, P, P],
        "bsa_aggregation_scores": [P, I, P, P, P, P, P],
        "bsa_rope_create": [ctypes.POINTER(P), P, ctypes.POINTER(RopeConfig)],
        "bsa_rope_destroy": [P],
        "bsa_rotary": [P, P, P, P, P, P, I, P],
        "bsa_cross_create": [ctypes.POINTER(P)] + [I] * 7 + [ctypes.c_double],
        "bsa_cross_destroy": [P],
        "bsa_cross_workspace_size": [P, ctypes.POINTER(Z), ctypes.POINTER(Z)],
        "bsa_cross_attention": [P] * 9 + [Z, P, P],
        "bsa_cross_attention_backward": [P] * 13 + [Z, P, P],
        "bsa_cross_check_status": [P, P],
        "bsa_cross_set_watchdog": [P, ctypes.c_longlong, I],
    }
    for name, args in sigs.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = I
    _lib = L
    return L


def _check(status: int):
    if status != 0:
        raise BsaError(status, load().bsa_last_error_string().decode())


def _ptr(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _params(p, heads):
    if isinstance(p, (int, float)):
        p = [float(p)] * heads
    arr = (ctypes.c_double * heads)(*[float(x) for x in p])
    if len(p) != heads:
        raise BsaError(1, f"expected {heads} per-head parameters, got {len(p)}")
    return arr


class Timings(ctypes.Structure):
    """bsa_timings_t: device milliseconds of the phases of one bsa_forward call."""
    _fields_ = [(n, ctypes.c_float) for n in ("summaries_ms", "select_ms", "pairing_ms",
                                               "attention_ms", "unpermute_ms", "total_ms")]

    def as_dict(self):
        return {n: float(getattr(self, n)) for n, _ in self._fields_}


class MaskUnion(ctypes.Structure):
    """bsa_mask_union_t: window (left, right) in blocks, sink tokens, intra rule."""
    _fields_ = [("window_left", ctypes.c_int), ("window_right", ctypes.c_int),
                ("sink_tokens", ctypes.c_longlong), ("intra_mode", ctypes.c_int),
                ("intra_param", ctypes.POINTER(ctypes.c_double))]


def mask_union(heads, window=(-1, -1), sink_tokens=0, intra_mode=0, intra_params=None):
    """A MaskUnion (kept alive with its per-head intra array)."""
    u = MaskUnion(int(window[0]), int(window[1]), int(sink_tokens), int(intra_mode), None)
    if intra_params is not None:
        arr = _params(intra_params, heads) if not isinstance(intra_params, (int, float)) \
            else _params([float(intra_params)] * heads, heads)
        u._keep = arr
        u.intra_param = ctypes.cast(arr, ctypes.POINTER(ctypes.c_double))
    return u


class RopeConfig(ctypes.Structure):
    """bsa_rope_config_t (axes in the order t, y, x)."""
    _fields_ = [("dim", ctypes.c_int * 3), ("layout", ctypes.c_int), ("scaling", ctypes.c_int),
                ("theta", ctypes.c_double), ("factor", ctypes.c_double * 3),
                ("orig_len", ctypes.c_double * 3), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double), ("mscale", ctypes.c_double),
                ("heads_k", ctypes.c_int)]


_ROPE_LAYOUT = {"interleaved": 0, "half": 1}
_ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


def _check_view(t, shape, dtype, device, name):
    """A strided tensor (bsa_view_t): its head dimension contiguous, the rest checked by the call."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise BsaError(1, f"{name} must be a tensor on {device}")
    if t.dtype != dtype or t.shape != shape or t.stride(3) != 1:
        raise BsaError(1, f"{name} must be a {dtype} tensor of shape {tuple(shape)} whose last axis is "
                          f"contiguous, got {t.dtype} {tuple(t.shape)} with strides {t.stride()}")


def _views(*tensors):
    """One bsa_view_t per tensor (None: zeros) and their addresses (None: NULL)."""
    flat = array.array("q")
    for t in tensors:
        if t is None:
            flat.extend((0, 0, 0, 0))
        else:
            b, n, h, _ = t.stride()
            flat.extend((t.data_ptr(), b, n, h))
    base = flat.buffer_info()[0]
    return flat, [None if t is None else base + 32 * i for i, t in enumerate(tensors)]


def _like(t):
    """An uninitialised contiguous tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _call(device, fn, *args):
    """fn(*args, the current stream of `device`) with that device current."""
    if torch.cuda.current_device() == device.index:
        _check(fn(*args, torch._C._cuda_getCurrentRawStream(device.index)))
    else:
        with torch.cuda.device(device):
            _check(fn(*args, torch._C._cuda_getCurrentRawStream(device.index)))


def _indexed(device):
    """`device` with its index (of the current device where it has none)."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


def _triple(x, kind=float):
    return (kind(x),) * 3 if isinstance(x, (int, float)) else tuple(kind(v) for v in x)


class Plan:
    """One attention problem: grid (T,H,W), block (bf,br,bc), heads, head_dim, text tokens."""

    def __init__(self, batch, T, H, W, bf, br, bc, heads, head_dim, n_text=0,
                 dtype=torch.bfloat16, device=None):
        L = load()
        if dtype not in _DT:
            raise BsaError(1, f"dtype must be float32 or bfloat16, got {dtype}")
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None \
            else torch.device(device)
        if self.device.type != "cuda":
            raise BsaError(1, "libbsa runs on CUDA devices only")
        self.dtype = dtype
        self._h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(L.bsa_plan_create(ctypes.byref(self._h), batch, T, H, W, bf, br, bc, heads,
                                     head_dim, n_text, _DT[dtype]))
        info = PlanInfo()
        _check(L.bsa_plan_get_info(self._h, ctypes.byref(info)))
        self.info = info

    def __del__(self):
        h = getattr(self, "_h", None)
        if h and _lib is not None:
            try:
                with torch.cuda.device(self.device):
                    _lib.bsa_plan_destroy(h)
            except Exception:
                pass
            self._h = None

    # ---------------------------------------------------------------- sizes
    @property
    def orig_shape(self):
        i = self.info
        return (i.batch, i.n_tot, i.heads, i.head_dim)

    @property
    def blk_shape(self):
        i = self.info
        return (i.batch, i.heads, i.npad_tot, i.head_dim)

    @property
    def cent_shape(self):
        i = self.info
        return (i.batch, i.heads, i.nb, i.head_dim)

    def kmax_for(self, mode, params) -> int:
        k = ctypes.c_int()
        _check(load().bsa_kmax_for(self._h, mode, _params(params, self.info.heads), ctypes.byref(k)))
        return k.value

    def workspace_size(self, kmax):
        a, b = ctypes.c_size_t(), ctypes.c_size_t()
        _check(load().bsa_workspace_size(self._h, kmax, ctypes.byref(a), ctypes.byref(b)))
        return a.value, b.value

    def _new(self, shape, dtype=None):
        return torch.empty(shape, dtype=dtype or self.dtype, device=self.device)

    def _check_tensor(self, t, shape, dtype=None, name="tensor"):
        dtype = dtype or self.dtype
        if not isinstance(t, torch.Tensor) or t.device != self.device:
            raise BsaError(1, f"{name} must be a tensor on {self.device}")
        if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise BsaError(1, f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, "
                              f"got {t.dtype} {tuple(t.shape)}")

    # ---------------------------------------------------------------- calls
    def permute(self, x, centroids=False, out=None):
        self._check_tensor(x, self.orig_shape, name="x")
        out = self._new(self.blk_shape) if out is None else out
        cent = self._new(self.cent_shape, torch.float32) if centroids else None
        _check(load().bsa_permute(self._h, _ptr(x), _ptr(out), _ptr(cent), _stream(self.device)))
        return (out, cent) if centroids else out

    def permute_qkv(self, q, k, v):
        for t, n in ((q, "q"), (k, "k"), (v, "v")):
            self._check_tensor(t, self.orig_shape, name=n)
        qb, kb, vb = (self._new(self.blk_shape) for _ in range(3))
        qc, kc = (self._new(self.cent_shape, torch.float32) for _ in range(2))
        _check(load().bsa_permute_qkv(self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(qb), _ptr(kb),
                                      _ptr(vb), _ptr(qc), _ptr(kc), _stream(self.device)))
        return qb, kb, vb, qc, kc

    def centroids(self, q, k):
        """Q and K block centroids straight from the original layout (bsa_centroids)."""
        self._check_tensor(q, self.orig_shape, name="q")
        self._check_tensor(k, self.orig_shape, name="k")
        qc, kc = (self._new(self.cent_shape, torch.float32) for _ in range(2))
        _check(load().bsa_centroids(self._h, _ptr(q), _ptr(k), _ptr(qc), _ptr(kc),
                                    _stream(self.device)))
        return qc, kc

    def sics(self, x, out=None):
        """Sum of intra-block cosine similarities per video block, [B,Hd,nb] fp32 (bsa_sics)."""
        self._check_tensor(x, self.orig_shape, name="x")
        i = self.info
        out = self._new((i.batch, i.heads, i.nb), torch.float32) if out is None else out
        self._check_tensor(out, (i.batch, i.heads, i.nb), torch.float32, "out")
        _check(load().bsa_sics(self._h, _ptr(x), _ptr(out), _stream(self.device)))
        return out

    def pair_tiles(self, idx, cnt):
        """bsa_pair_tiles: the pairing workspace (a uint8 tensor) for these lists."""
        z = ctypes.c_size_t()
        kmax = idx.shape[-1]
        _check(load().bsa_pair_workspace_size(self._h, kmax, ctypes.byref(z)))
        ws = self._new((max(z.value, 1),), torch.uint8)
        _check(load().bsa_pair_tiles(self._h, _ptr(idx), _ptr(cnt), kmax, _ptr(ws), ws.numel(),
                                     _stream(self.device)))
        return ws

    def attention_paired(self, q, k, v, idx, cnt, ws, out=None, dev_status=None):
        """bsa_attention_paired on the schedule of pair_tiles(idx, cnt)."""
        for t, n in ((q, "q"), (k, "k"), (v, "v")):
            self._check_tensor(t, self.orig_shape, name=n)
        out = self._new(self.orig_shape) if out is None else out
        _check(load().bsa_attention_paired(self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(idx), _ptr(cnt),
                                           idx.shape[-1], _ptr(ws), ws.numel(), _ptr(out),
                                           _ptr(dev_status), _stream(self.device)))
        return out

    def attention_orig(self, q, k, v, idx, cnt, out=None, dev_status=None):
        """Attention on the original layout; the layout transform is fused (bsa_attention_orig)."""
        for t, n in ((q, "q"), (k, "k"), (v, "v")):
            self._check_tensor(t, self.orig_shape, name=n)
        i = self.info
        kmax = idx.shape[-1]
        self._check_tensor(idx, (i.batch, i.heads, i.nb, kmax), torch.int32, "idx")
        self._check_tensor(cnt, (i.batch, i.heads, i.nb), torch.int32, "cnt")
        out = self._new(self.orig_shape) if out is None else out
        _check(load().bsa_attention_orig(self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(idx), _ptr(cnt),
                                         kmax, _ptr(out), _ptr(dev_status), _stream(self.device)))
        return out

    def unpermute(self, o_blk, out=None):
        self._check_tensor(o_blk, self.blk_shape, name="o_blk")
        out = self._new(self.orig_shape) if out is None else out
        _check(load().bsa_unpermute(self._h, _ptr(o_blk), _ptr(out), _stream(self.device)))
        return out

    def _lists(self, kmax):
        i = self.info
        return (self._new((i.batch, i.heads, i.nb, kmax), torch.int32),
                self._new((i.batch, i.heads, i.nb), torch.int32))

    def select(self, q_blk, k_blk, mode, params, kmax=None, scores=False):
        self._check_tensor(q_blk, self.blk_shape, name="q_blk")
        self._check_tensor(k_blk, self.blk_shape, name="k_blk")
        kmax = self.kmax_for(mode, params) if kmax is None else kmax
        idx, cnt = self._lists(kmax)
        i = self.info
        sc = self._new((i.batch, i.heads, i.nb, i.nb), torch.float32) if scores else None
        ws = self._new((max(self.workspace_size(kmax)[0], 1),), torch.uint8)
        _check(load().bsa_select(self._h, _ptr(q_blk), _ptr(k_blk), mode,
                                 _params(params, i.heads), kmax, _ptr(idx), _ptr(cnt), _ptr(sc),
                                 _ptr(ws), ws.numel(), _stream(self.device)))
        return (idx, cnt, sc) if scores else (idx, cnt)

    def select_centroids(self, q_cent, k_cent, mode, params, kmax=None, scores=False):
        self._check_tensor(q_cent, self.cent_shape, torch.float32, "q_cent")
        self._check_tensor(k_cent, self.cent_shape, torch.float32, "k_cent")
        kmax = self.kmax_for(mode, params) if kmax is None else kmax
        idx, cnt = self._lists(kmax)
        i = self.info
        sc = self._new((i.batch, i.heads, i.nb, i.nb), torch.float32) if scores else None
        _check(load().bsa_select_centroids(self._h, _ptr(q_cent), _ptr(k_cent), mode,
                                           _params(params, i.heads), kmax, _ptr(idx), _ptr(cnt),
                                           _ptr(sc), _stream(self.device)))
        return (idx, cnt, sc) if scores else (idx, cnt)

    def attention(self, q_blk, k_blk, v_blk, idx, cnt, out=None, dev_status=None):
        for t, n in ((q_blk, "q_blk"), (k_blk, "k_blk"), (v_blk, "v_blk")):
            self._check_tensor(t, self.blk_shape, name=n)
        i = self.info
        kmax = idx.shape[-1]
        self._check_tensor(idx, (i.batch, i.heads, i.nb, kmax), torch.int32, "idx")
        self._check_tensor(cnt, (i.batch, i.heads, i.nb), torch.int32, "cnt")
        out = self._new(self.blk_shape) if out is None else out
        _check(load().bsa_attention(self._h, _ptr(q_blk), _ptr(k_blk), _ptr(v_blk), _ptr(idx),
                                    _ptr(cnt), kmax, _ptr(out), _ptr(dev_status),
                                    _stream(self.device)))
        return out

    def forward(self, q, k, v, mode, params, kmax=None, out=None, workspace=None,
                return_lists=False):
        for t, n in ((q, "q"), (k, "k"), (v, "v")):
            self._check_tensor(t, self.orig_shape, name=n)
        kmax = self.kmax_for(mode, params) if kmax is None else kmax
        out = self._new(self.orig_shape) if out is None else out
        need = self.workspace_size(kmax)[1]
        ws = self._new((need,), torch.uint8) if workspace is None else workspace
        idx, cnt = self._lists(kmax) if return_lists else (None, None)
        _check(load().bsa_forward(self._h, _ptr(q), _ptr(k), _ptr(v), mode,
                                  _params(params, self.info.heads), kmax, _ptr(out), _ptr(idx),
                                  _ptr(cnt), _ptr(ws), ws.numel(), None, _stream(self.device)))
        return (out, idx, cnt) if return_lists else out

    def forward_timed(self, q, k, v, mode, params, kmax=None, out=None, workspace=None):
        """bsa_forward_timed: the forward plus the device time of each phase
        (synchronises); returns (out, dict of milliseconds)."""
        for t, n in ((q, "q"), (k, "k"), (v, "v")):
            self._check_tensor(t, self.orig_shape, name=n)
        kmax = self.kmax_for(mode, params) if kmax is None else kmax
        out = self._new(self.orig_shape) if out is None else out
        need = self.workspace_size(kmax)[1]
        ws = self._new((need,), torch.uint8) if workspace is None else workspace
        t = Timings()
        _check(load().bsa_forward_timed(self._h, _ptr(q), _ptr(k), _ptr(v), mode,
                                        _params(params, self.info.heads), kmax, _ptr(out), None,
                                        None, _ptr(ws), ws.numel(), None, _stream(self.device),
                                        ctypes.byref(t)))
        return out, t.as_dict()

    # ------------------------------------------------------ rotary positions
    def rope(self, dims, theta=10000.0, layout="interleaved", scaling="none", factor=1.0,
             orig_len=None, beta_fast=32.0, beta_slow=1.0, mscale=1.0, heads_k=None) -> "Rope":
        """Rotary positions over this plan's grid (bsa_rope_create): dims = rotated elements of
        the t, y and x axis; layout "interleaved" or "half"; scaling "none", "linear", "ntk" or
        "yarn" by factor (one number or one per axis; "yarn" also takes the trained orig_len);
        heads_k = heads of K where it has fewer than Q."""
        return Rope(self, dims, theta, layout, scaling, factor, orig_len, beta_fast, beta_slow,
                    mscale, heads_k)

    def cross(self, n_kv, heads_kv=None, scale=None) -> "CrossAttention":
        """Cross attention from this plan's tokens (video, then text) to n_kv encoder states."""
        i = self.info
        return CrossAttention(i.batch, i.n_tot, n_kv, i.heads, heads_kv, i.head_dim, self.dtype,
                              scale, self.device)

    # --------------------------------------------------------- mask union
    def kmax_for_union(self, mode, params, union) -> int:
        k = ctypes.c_int()
        _check(load().bsa_kmax_for_union(self._h, mode, _params(params, self.info.heads),
                                         ctypes.byref(union) if union is not None else None,
                                         ctypes.byref(k)))
        return k.value

    def union_workspace_size(self, kmax, union):
        a, b = ctypes.c_size_t(), ctypes.c_size_t()
        _check(load().bsa_union_workspace_size(self._h, kmax,
                                               ctypes.byref(union) if union is not None else None,
                                               ctypes.byref(a), ctypes.byref(b)))
        return a.value, b.value

    def select_union(self, q_cent, k_cent, mode, params, union, intra_scores=None, kmax=None,
                     scores=False):
        """bsa_select_union: Top-K/Top-P lists united with window, sink and intra blocks."""
        i = self.info
        self._check_tensor(q_cent, self.cent_shape, torch.float32, "q_cent")
        self._check_tensor(k_cent, self.cent_shape, torch.float32, "k_cent")
        if intra_scores is not None:
            self._check_tensor(intra_scores, (i.batch, i.heads, i.nb), torch.float32, "intra_scores")
        kmax = kmax or self.kmax_for_union(mode, params, union)
        idx, cnt = self._lists(kmax)
        sc = self._new((i.batch, i.heads, i.nb, i.nb), torch.float32) if scores else None
        sel_ws, _ = self.union_workspace_size(kmax, union)
        ws = self._new((max(sel_ws, 1),), torch.uint8)
        _check(load().bsa_select_union(self._h, _ptr(q_cent), _ptr(k_cent), mode,
                                       _params(params, i.heads), ctypes.byref(union),
                                       _ptr(intra_scores), kmax, _ptr(idx), _ptr(cnt), _ptr(sc),
                                       _ptr(ws), ws.numel(), _stream(self.device)))
        return (idx, cnt, sc) if scores else (idx, cnt)

    def forward_union(self, q, k, v, mode, params, union, kmax=None, out=None, workspace=None,
                      dev_status=None):
        """bsa_forward_union: the whole path with the mask union; returns (o, idx, cnt)."""
        for t, n in ((q, "q"), (k, "k"), (v, "v")):
            self._check_tensor(t, self.orig_shape, name=n)
        kmax = kmax or self.kmax_for_union(mode, params, union)
        idx, cnt = self._lists(kmax)
        out = self._new(self.orig_shape) if out is None else out
        _, fwd_ws = self.union_workspace_size(kmax, union)
        ws = workspace if workspace is not None else self._new((max(fwd_ws, 1),), torch.uint8)
        _check(load().bsa_forward_union(self._h, _ptr(q), _ptr(k), _ptr(v), mode,
                                        _params(params, self.info.heads),
                                        ctypes.byref(union) if union is not None else None, kmax,
                                        _ptr(out), _ptr(idx), _ptr(cnt), _ptr(ws), ws.numel(),
                                        _ptr(dev_status), _stream(self.device)))
        return out, idx, cnt

    # ---------------------------------------------------- box estimators
    @property
    def box_shape(self):
        i = self.info
        return (i.batch, i.heads, i.nb, i.head_dim, 2)

    def box_summaries(self, q, k):
        """(max, min) per video block and dimension of Q and K (bsa_box_summaries)."""
        self._check_tensor(q, self.orig_shape, name="q")
        self._check_tensor(k, self.orig_shape, name="k")
        qb, kb = (self._new(self.box_shape, torch.float32) for _ in range(2))
        _check(load().bsa_box_summaries(self._h, _ptr(q), _ptr(k), _ptr(qb), _ptr(kb),
                                        _stream(self.device)))
        return qb, kb

    def select_box(self, est, q_box, k_box, mode, params, union=None, intra_scores=None,
                   kmax=None, scores=False):
        """bsa_select_box: lists from the DSA (est 1) or DSA2 (est 2) estimator."""
        i = self.info
        self._check_tensor(q_box, self.box_shape, torch.float32, "q_box")
        self._check_tensor(k_box, self.box_shape, torch.float32, "k_box")
        kmax = kmax or self.kmax_for_union(mode, params, union)
        idx, cnt = self._lists(kmax)
        sc = self._new((i.batch, i.heads, i.nb, i.nb), torch.float32) if scores else None
        sel_ws = self.union_workspace_size(kmax, union)[0] if union is not None else 0
        ws = self._new((max(sel_ws, 1),), torch.uint8)
        _check(load().bsa_select_box(self._h, est, _ptr(q_box), _ptr(k_box), mode,
                                     _params(params, i.heads),
                                     ctypes.byref(union) if union is not None else None,
                                     _ptr(intra_scores), kmax, _ptr(idx), _ptr(cnt), _ptr(sc),
                                     _ptr(ws), ws.numel(), _stream(self.device)))
        return (idx, cnt, sc) if scores else (idx, cnt)

    def forward_estimator(self, q, k, v, est, mode, params, union=None, kmax=None, out=None,
                          dev_status=None):
        """bsa_forward_estimator: the whole path with MEAN / DSA / DSA2; returns (o, idx, cnt)."""
        for t, n in ((q, "q"), (k, "k"), (v, "v")):
            self._check_tensor(t, self.orig_shape, name=n)
        kmax = kmax or self.kmax_for_union(mode, params, union)
        idx, cnt = self._lists(kmax)
        out = self._new(self.orig_shape) if out is None else out
        z = ctypes.c_size_t()
        u = ctypes.byref(union) if union is not None else None
        _check(load().bsa_estimator_workspace_size(self._h, est, kmax, u, ctypes.byref(z)))
        ws = self._new((max(z.value, 1),), torch.uint8)
        _check(load().bsa_forward_estimator(self._h, _ptr(q), _ptr(k), _ptr(v), est, mode,
                                            _params(params, self.info.heads), u, kmax, _ptr(out),
                                            _ptr(idx), _ptr(cnt), _ptr(ws), ws.numel(),
                                            _ptr(dev_status), _stream(self.device)))
        return out, idx, cnt

    def check_status(self):
        """Synchronise the current stream and raise if a kernel recorded an error."""
        _check(load().bsa_check_status(self._h, _stream(self.device)))

    def set_watchdog(self, wait_limit_cycles=0, withhold_copy=0):
        """Bound of the attention kernel's in-kernel waits (0 = default, about a
        second) and the timeout path's test hook (bsa_plan_set_watchdog)."""
        _check(load().bsa_plan_set_watchdog(self._h, int(wait_limit_cycles), int(withhold_copy)))


class Rope:
    """Rotary positions of one plan's tokens; made by Plan.rope."""

    def __init__(self, plan, dims, theta, layout, scaling, factor, orig_len, beta_fast, beta_slow,
                 mscale, heads_k):
        if layout not in _ROPE_LAYOUT or scaling not in _ROPE_SCALING:
            raise BsaError(1, f"unknown rope layout {layout!r} or scaling {scaling!r}")
        dims, factor, orig_len = _triple(dims, int), _triple(factor), _triple(orig_len or 0.0)
        if not (len(dims) == len(factor) == len(orig_len) == 3):
            raise BsaError(1, "dims, factor and orig_len take one value or one per axis (t, y, x)")
        i = plan.info
        c = RopeConfig((ctypes.c_int * 3)(*dims), _ROPE_LAYOUT[layout], _ROPE_SCALING[scaling],
                       float(theta), (ctypes.c_double * 3)(*factor), (ctypes.c_double * 3)(*orig_len),
                       float(beta_fast), float(beta_slow), float(mscale), int(heads_k or 0))
        self.device, self.dtype = _indexed(plan.device), plan.dtype
        self.q_shape = torch.Size(plan.orig_shape)
        self.k_shape = torch.Size((i.batch, i.n_tot, heads_k or i.heads, i.head_dim))
        self._h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(load().bsa_rope_create(ctypes.byref(self._h), plan._h, ctypes.byref(c)))

    def __del__(self):
        h = getattr(self, "_h", None)
        if h and _lib is not None:
            _lib.bsa_rope_destroy(h)
            self._h = None

    def apply(self, q, k=None, t_origin=None, out=None):
        """Rotates q [B,Ntot,heads,D] and k [B,Ntot,heads_k,D] (strided views are fine).

        t_origin: int64 [B], added to t.  out: (q_out, k_out), or one tensor without k; the
        inputs themselves for a rotation in place.  Returns (q_out, k_out), or q_out without k."""
        return self._run(q, k, t_origin, out, 0)

    def backward(self, dq, dk=None, t_origin=None, out=None):
        """The gradients of apply's inputs from those of its outputs (the transposed rotation)."""
        return self._run(dq, dk, t_origin, out, 1)

    def _run(self, q, k, t_origin, out, backward):
        dev, dt = self.device, self.dtype
        _check_view(q, self.q_shape, dt, dev, "q")
        if k is not None:
            _check_view(k, self.k_shape, dt, dev, "k")
        if t_origin is not None and (not isinstance(t_origin, torch.Tensor) or
                                     t_origin.dtype != torch.int64 or t_origin.device != dev or
                                     t_origin.shape != self.q_shape[:1] or
                                     not t_origin.is_contiguous()):
            raise BsaError(1, f"t_origin must be an int64 tensor of shape {tuple(self.q_shape[:1])} on {dev}")
        if out is None:
            qo = _like(q)
            ko = None if k is None else _like(k)
        else:
            qo, ko = out if k is not None else (out, None)
            _check_view(qo, self.q_shape, dt, dev, "q_out")
            if k is not None:
                _check_view(ko, self.k_shape, dt, dev, "k_out")
        keep, v = _views(q, k, qo, ko)
        _call(dev, load().bsa_rotary, self._h, *v, None if t_origin is None else t_origin.data_ptr(),
              backward)
        return qo if k is None else (qo, ko)


class CrossAttention:
    """Cross attention from n_q query tokens to n_kv encoder states (bsa_cross_create).

    q, o [B,n_q,heads,D]; k, v [B,n_kv,heads_kv,D] (strided views are fine).  kv_len: int32 [B],
    keys of each batch element; key_mask: bool or uint8 [B,n_kv], False at padding."""

    def __init__(self, batch, n_q, n_kv, heads, heads_kv=None, head_dim=128, dtype=torch.bfloat16,
                 scale=None, device=None):
        L = load()
        if dtype not in _DT:
            raise BsaError(1, f"dtype must be float32 or bfloat16, got {dtype}")
        self.device = _indexed(device)
        if self.device.type != "cuda":
            raise BsaError(1, "libbsa runs on CUDA devices only")
        if scale is not None and not scale > 0.0:
            raise BsaError(1, f"scale must be above 0, got {scale}")
        heads_kv = heads if heads_kv is None else heads_kv
        self.dtype = dtype
        self._h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(L.bsa_cross_create(ctypes.byref(self._h), batch, n_q, n_kv, heads, heads_kv,
                                      head_dim, _DT[dtype], float(scale or 0.0)))
        self.q_shape = torch.Size((batch, n_q, heads, head_dim))
        self.kv_shape = torch.Size((batch, n_kv, heads_kv, head_dim))
        self.lse_shape = torch.Size((batch, heads, n_q))
        f, b = ctypes.c_size_t(), ctypes.c_size_t()
        _check(L.bsa_cross_workspace_size(self._h, ctypes.byref(f), ctypes.byref(b)))
        self.forward_ws, self.backward_ws = f.value, b.value

    def __del__(self):
        h = getattr(self, "_h", None)
        if h and _lib is not None:
            try:
                with torch.cuda.device(self.device):
                    _lib.bsa_cross_destroy(h)
            except Exception:
                pass
            self._h = None

    def _view(self, t, kv, name):
        _check_view(t, self.kv_shape if kv else self.q_shape, self.dtype, self.device, name)

    def _masks(self, kv_len, key_mask):
        for t, shape, types, name in ((kv_len, self.kv_shape[:1], (torch.int32,), "kv_len"),
                                      (key_mask, self.kv_shape[:2], (torch.bool, torch.uint8), "key_mask")):
            if t is not None and (not isinstance(t, torch.Tensor) or t.device != self.device or
                                  t.dtype not in types or t.shape != shape or not t.is_contiguous()):
                raise BsaError(1, f"{name} must be a contiguous {types[0]} tensor of shape "
                                  f"{tuple(shape)} on {self.device}")
        return (None if kv_len is None else kv_len.data_ptr(),
                None if key_mask is None else key_mask.data_ptr())

    def _workspace(self, ws, need, dev_status):
        for t, types, name in ((ws, None, "workspace"), (dev_status, torch.int32, "dev_status")):
            if t is not None and (not isinstance(t, torch.Tensor) or t.device != self.device or
                                  not t.is_contiguous() or (types and (t.dtype != types or not t.numel()))):
                raise BsaError(1, f"{name} must be a contiguous {f'{types} ' if types else ''}tensor on {self.device}")
        if ws is None and need:
            ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size()), ws

    def _lse(self, lse):
        if not isinstance(lse, torch.Tensor) or lse.device != self.device or \
                lse.dtype != torch.float32 or lse.shape != self.lse_shape or not lse.is_contiguous():
            raise BsaError(1, f"lse must be a contiguous float32 tensor of shape {tuple(self.lse_shape)} "
                              f"on {self.device}")

    def forward(self, q, k, v, kv_len=None, key_mask=None, out=None, return_lse=False,
                workspace=None, dev_status=None):
        """O = softmax(scale Q K^T) V; with return_lse also the log-sum-exp of every row
        (float32 [B,heads,n_q]), which backward takes."""
        self._view(q, False, "q")
        self._view(k, True, "k")
        self._view(v, True, "v")
        if out is None:
            out = _like(q)
        else:
            self._view(out, False, "o")
        lse = torch.empty(self.lse_shape, dtype=torch.float32, device=self.device) if return_lse else None
        keep, views = _views(q, k, v, out)
        masks = self._masks(kv_len, key_mask)
        ws, keep_ws = self._workspace(workspace, self.forward_ws, dev_status)
        _call(self.device, load().bsa_cross_attention, self._h, *views[:3], *masks, views[3],
              None if lse is None else lse.data_ptr(), *ws,
              None if dev_status is None else dev_status.data_ptr())
        return (out, lse) if return_lse else out

    def backward(self, d_o, q, k, v, o, lse, kv_len=None, key_mask=None, out=None, workspace=None,
                 dev_status=None):
        """(dq, dk, dv) from d_o, the forward's inputs and its outputs o and lse; out: the three
        tensors to write."""
        for t, kv, name in ((d_o, False, "d_o"), (q, False, "q"), (k, True, "k"), (v, True, "v"),
                            (o, False, "o")):
            self._view(t, kv, name)
        self._lse(lse)
        if out is None:
            out = (_like(q), _like(k), _like(v))
        else:
            for t, kv, name in zip(out, (False, True, True), ("dq", "dk", "dv")):
                self._view(t, kv, name)
        dq, dk, dv = out
        keep, views = _views(q, k, v, o, d_o, dq, dk, dv)
        masks = self._masks(kv_len, key_mask)
        ws, keep_ws = self._workspace(workspace, self.backward_ws, dev_status)
        _call(self.device, load().bsa_cross_attention_backward, self._h, *views[:3], *masks, views[3],
              lse.data_ptr(), *views[4:], *ws, None if dev_status is None else dev_status.data_ptr())
        return dq, dk, dv

    def check_status(self):
        """Synchronise the current stream and raise if a kernel recorded an error."""
        _call(self.device, load().bsa_cross_check_status, self._h)

    def set_watchdog(self, wait_limit_cycles=0, withhold_copy=0):
        """Bound of the tensor-core kernels' waits (0 = default, about a second) and the timeout
        path's test hook (bsa_cross_set_watchdog)."""
        _check(load().bsa_cross_set_watchdog(self._h, int(wait_limit_cycles), int(withhold_copy)))


def aggregation_scores(plans, x):
    """Aggregation evaluation over candidate blocking schemes (bsa_aggregation_scores).

    plans: 1..8 Plans that differ only in block shape.  Returns (sics, as_, choice):
    sics[c] [B,Hd,nb_c] fp32, as_ [n,B,Hd] float64, choice [B,Hd] int32.
    """
    plans = list(plans)
    n = len(plans)
    p0 = plans[0]
    p0._check_tensor(x, p0.orig_shape, name="x")
    i = p0.info
    sics = [p._new((i.batch, i.heads, p.info.nb), torch.float32) for p in plans]
    as_ = p0._new((n, i.batch, i.heads), torch.float64)
    choice = p0._new((i.batch, i.heads), torch.int32)
    handles = (ctypes.c_void_p * n)(*[p._h.value for p in plans])
    outs = (ctypes.c_void_p * n)(*[t.data_ptr() for t in sics])
    _check(load().bsa_aggregation_scores(handles, n, _ptr(x), outs, _ptr(as_), _ptr(choice),
                                         _stream(p0.device)))
    return sics, as_, choice


def forward_grouped(plans, head_plan, q, k, v, mode, params, union=None, kmax=None, out=None):
    """bsa_forward_grouped: each (b, h) served by plans[head_plan[b*Hd + h]].

    head_plan: sequence or int tensor of B*Hd plan indices (host values).
    Returns (o, lists) with lists[c] = (idx, cnt) of plan c (only its heads written).
    """
    plans = list(plans)
    n = len(plans)
    p0 = plans[0]
    for t, nm in ((q, "q"), (k, "k"), (v, "v")):
        p0._check_tensor(t, p0.orig_shape, name=nm)
    hp = [int(x) for x in (head_plan.flatten().tolist() if isinstance(head_plan, torch.Tensor)
                           else head_plan)]
    hp_arr = (ctypes.c_int32 * len(hp))(*hp)
    kmaxes = kmax or [p.kmax_for_union(mode, params, union) for p in plans]
    km_arr = (ctypes.c_int * n)(*kmaxes)
    lists = [p._lists(km) for p, km in zip(plans, kmaxes)]
    for idx, cnt in lists:
        cnt.zero_()
    idx_arr = (ctypes.c_void_p * n)(*[l[0].data_ptr() for l in lists])
    cnt_arr = (ctypes.c_void_p * n)(*[l[1].data_ptr() for l in lists])
    handles = (ctypes.c_void_p * n)(*[p._h.value for p in plans])
    u = ctypes.byref(union) if union is not None else None
    z = ctypes.c_size_t()
    _check(load().bsa_grouped_workspace_size(handles, n, km_arr, u, ctypes.byref(z)))
    ws = p0._new((max(z.value, 1),), torch.uint8)
    out = p0._new(p0.orig_shape) if out is None else out
    _check(load().bsa_forward_grouped(handles, n, hp_arr, _ptr(q), _ptr(k), _ptr(v), mode,
                                      _params(params, p0.info.heads), u, km_arr, _ptr(out),
                                      idx_arr, cnt_arr, _ptr(ws), ws.numel(), None,
                                      _stream(p0.device)))
    return out, lists


def plan_for(w, device=None) -> Plan:
    """A Plan for a synthetic Workload-like object (attributes B,T,H,W,bf,br,bc,Hd,D,n_text,dtype)."""
    dt = torch.float32 if w.dtype == "f32" else torch.bfloat16
    return Plan(w.B, w.T, w.H, w.W, w.bf, w.br, w.bc, w.Hd, w.D, w.n_text, dt, device)

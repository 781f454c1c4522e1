"""Thin torch binding of the TurboQuant C ABI (argument marshalling only).

Every step of encode, dequant and decode attention runs in the CUDA kernels
of libtq_b200.so; torch supplies device memory, strides and the current
stream.  The names follow the C ABI (include/tq.h).
"""

import ctypes
import math
from dataclasses import dataclass
from typing import Optional

import numpy as np
import torch

from . import _lib as L

_DTYPES = {torch.float32: L.TQ_F32, torch.bfloat16: L.TQ_BF16, torch.float16: L.TQ_F16}


# the handle of a device's current stream, without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """What a call on `stream` (None: the current one) returns.  The memory
    belongs to that stream: none that another one still works on, and none
    that another one gets while the call runs."""
    if stream is None or stream.cuda_stream == _raw_stream(torch.cuda.current_device() if device.index is None
                                                           else device.index):
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream)
                           else torch.cuda.ExternalStream(stream.cuda_stream, device)):
        return torch.empty(shape, dtype=dtype, device=device)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------- host calls

def make_codebook(d: int, bits_mse: int, dist: str = "gauss"):
    """(centroids, thresholds) as numpy fp32 arrays from tq_make_codebook."""
    K = 1 << bits_mse
    c = (ctypes.c_float * K)()
    t = (ctypes.c_float * max(K - 1, 1))()
    L.check(L.lib().tq_make_codebook(d, bits_mse, L.TQ_CB_BETA if dist == "beta" else L.TQ_CB_GAUSS, c, t))
    return np.frombuffer(c, np.float32).copy(), np.frombuffer(t, np.float32)[: K - 1].copy()


def make_signs(seed: int, d: int) -> np.ndarray:
    s = np.empty(d, np.int8)
    L.check(L.lib().tq_make_signs(seed, d, s.ctypes.data))
    return s


def make_qjl(seed: int, d: int) -> np.ndarray:
    S = np.empty((d, d), np.float32)
    L.check(L.lib().tq_make_qjl(seed, d, S.ctypes.data_as(ctypes.POINTER(ctypes.c_float))))
    return S


def make_rotation(seed: int, d: int) -> np.ndarray:
    """Dense Haar rotation Pi (tq_make_rotation), numpy fp32 [d, d]."""
    R = np.empty((d, d), np.float32)
    L.check(L.lib().tq_make_rotation(seed, d, R.ctypes.data_as(ctypes.POINTER(ctypes.c_float))))
    return R


def code_bytes(d: int, bits: int, variant: str) -> int:
    return int(L.lib().tq_code_bytes(d, bits, L.TQ_PROD if variant == "prod" else L.TQ_MSE))


def qjl_bytes(d: int, variant: str) -> int:
    return int(L.lib().tq_qjl_bytes(d, L.TQ_PROD if variant == "prod" else L.TQ_MSE))


# ------------------------------------------------------------ quantizer

class Quantizer:
    """Device-resident parameters of one TurboQuant quantizer."""

    def __init__(self, d: int, bits: int, variant: str = "mse", seed_rot: int = 0,
                 seed_qjl: int = 1, dist: str = "gauss", device="cuda", rotation: str = "hadamard",
                 channels: Optional[torch.Tensor] = None):
        assert variant in ("mse", "prod") and rotation in ("hadamard", "dense")
        self.d, self.bits, self.variant = d, bits, variant
        self.seed_rot, self.seed_qjl, self.dist, self.rotation = seed_rot, seed_qjl, dist, rotation
        self.bm = bits - 1 if variant == "prod" else bits
        dev = torch.device(device)
        if self.bm > 0:
            c, t = make_codebook(d, self.bm, dist)
            self.centroids = torch.from_numpy(c).to(dev)
            self.thresholds = torch.from_numpy(t).to(dev) if t.size else torch.zeros(1, device=dev)
        else:
            self.centroids = self.thresholds = None
        self.signs = torch.from_numpy(make_signs(seed_rot, d)).to(dev)
        self.S = torch.from_numpy(make_qjl(seed_qjl, d)).to(dev) if variant == "prod" else None
        self.rot = torch.from_numpy(make_rotation(seed_rot, d)).to(dev) if rotation == "dense" else None
        self.channels = None if channels is None else channels.to(device=dev, dtype=torch.int32).contiguous()
        self._c = L.TqQuantizer(d, bits, L.TQ_PROD if variant == "prod" else L.TQ_MSE,
                                L.TQ_ROT_DENSE if rotation == "dense" else L.TQ_ROT_HADAMARD,
                                _ptr(self.centroids), _ptr(self.thresholds), _ptr(self.signs), _ptr(self.S),
                                _ptr(self.rot), _ptr(self.channels))
        self._ref = ctypes.byref(self._c)

    @property
    def prod(self) -> bool:
        return self.variant == "prod"

    @property
    def code_bytes(self) -> int:
        return self.d * self.bm // 8

    @property
    def qjl_bytes(self) -> int:
        return self.d // 8 if self.prod else 0

    @property
    def record_bytes(self) -> int:
        """Stored bytes per vector: codes + sketch + fp32 norms."""
        return self.code_bytes + self.qjl_bytes + 4 + (4 if self.prod else 0)

    def c_struct(self) -> L.TqQuantizer:
        return self._c

    def c_ref(self):
        return self._ref


@dataclass
class PackedCache:
    """Packed records shaped [B, H, N, ...] (any strides over B, H, N)."""
    codes: Optional[torch.Tensor]
    norms: torch.Tensor
    qjl: Optional[torch.Tensor] = None
    rnorms: Optional[torch.Tensor] = None

    @property
    def shape(self):
        return tuple(self.norms.shape)

    def view(self) -> L.TqCacheView:
        # built once per (arrays, layout): a decode step passes the same views
        c, q, n, r = self.codes, self.qjl, self.norms, self.rnorms
        key = (None if c is None else c.data_ptr(), None if q is None else q.data_ptr(), n.data_ptr(),
               None if r is None else r.data_ptr(), n.stride())
        cached = self.__dict__.get("_view")
        if cached is not None and cached[0] == key:
            return cached[1]
        sb, sh, sn = key[4]
        for t in (self.codes, self.qjl, self.rnorms):
            if t is not None:
                w = t.shape[3] if t.dim() == 4 else 1
                assert t.stride()[:3] == (sb * w, sh * w, sn * w) and (t.dim() < 4 or w <= 1 or t.stride(3) == 1), \
                    "all arrays must share one record layout"
        v = L.TqCacheView(key[0], key[1], key[2], key[3], sb, sh, sn)
        self.__dict__["_view"] = (key, v, ctypes.byref(v))
        return v

    def c_ref(self):
        self.view()
        return self.__dict__["_view"][2]

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.codes, self.qjl, self.norms, self.rnorms)
                   if t is not None)


def empty_cache(qz: Quantizer, B: int, H: int, N: int, device="cuda", stream=None) -> PackedCache:
    """An uninitialised cache of B x H x N records, for use on `stream`."""
    dev = torch.device(device)

    def empty(*last, dtype):
        return _empty((B, H, N, *last), dtype, dev, stream)
    codes = empty(qz.code_bytes, dtype=torch.uint8) if qz.bm > 0 else None
    qjl = empty(qz.qjl_bytes, dtype=torch.uint8) if qz.prod else None
    rn = empty(dtype=torch.float32) if qz.prod else None
    return PackedCache(codes, empty(dtype=torch.float32), qjl, rn)


def _as_bhn(x: torch.Tensor) -> torch.Tensor:
    if x.dim() == 2:
        return x[None, None]
    if x.dim() == 3:
        return x[None]
    return x


# ------------------------------------------------------------- device calls

def encode(qz: Quantizer, x: torch.Tensor, out: Optional[PackedCache] = None, stream=None) -> PackedCache:
    """tq_encode of x shaped [B, H, N, d] (or [H, N, d] / [N, d]); the last
    dim must be contiguous; out defaults to a new [B, H, N] cache."""
    x4 = _as_bhn(x)
    B, H, N, d = x4.shape
    # a channel-group quantizer reads its channels of a wider row
    assert (d == qz.d if qz.channels is None else d >= qz.d) and x4.stride(3) == 1 and x4.dtype in _DTYPES
    if out is None:
        out = empty_cache(qz, B, H, N, x.device, stream)
    v = out.view()
    L.check(L.lib().tq_encode(ctypes.byref(qz.c_struct()), x4.data_ptr(), _DTYPES[x4.dtype], B, H, N,
                              x4.stride(0), x4.stride(1), x4.stride(2), ctypes.byref(v), _stream(stream)))
    return out


def dequant(qz: Quantizer, cache: PackedCache, stream=None) -> torch.Tensor:
    """tq_dequant into a new fp32 tensor [B, H, N, d]."""
    B, H, N = cache.shape
    out = _empty((B, H, N, qz.d), torch.float32, cache.norms.device, stream)
    v = cache.view()
    L.check(L.lib().tq_dequant(ctypes.byref(qz.c_struct()), ctypes.byref(v), B, H, N, out.data_ptr(),
                               _stream(stream)))
    return out


def decode_workspace_bytes(B: int, Hq: int, Hkv: int, seq_len: int, d: int) -> int:
    return int(L.lib().tq_decode_workspace_bytes(B, Hq, Hkv, seq_len, d))


class DecodeAttention:
    """Reusable tq_decode_attention call with its workspace allocated once
    (so that repeated steps allocate nothing)."""

    def __init__(self, kq: Quantizer, vq: Quantizer, B: int, Hq: int, Hkv: int, seq_len: int,
                 device="cuda"):
        self.kq, self.vq = kq, vq
        self.B, self.Hq, self.Hkv, self.seq_len = B, Hq, Hkv, seq_len
        nb = decode_workspace_bytes(B, Hq, Hkv, seq_len, kq.d)
        self.workspace = torch.empty(max(nb, 16), dtype=torch.uint8, device=device)
        self.ws_bytes = nb
        self.out = torch.empty((B, Hq, kq.d), dtype=torch.float32, device=device)

    def __call__(self, q: torch.Tensor, kcache: PackedCache, vcache: PackedCache, scale: Optional[float] = None,
                 seq_lens: Optional[torch.Tensor] = None, scores: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        B, Hq, d = q.shape
        assert (B, Hq) == (self.B, self.Hq) and q.is_contiguous() and q.dtype in _DTYPES
        if scale is None:
            scale = 1.0 / math.sqrt(d)
        out = self.out if out is None else out
        kv, vv = kcache.view(), vcache.view()
        if seq_lens is not None:
            assert seq_lens.dtype == torch.int32 and seq_lens.is_contiguous()
        L.check(L.lib().tq_decode_attention(
            ctypes.byref(self.kq.c_struct()), ctypes.byref(self.vq.c_struct()), q.data_ptr(), _DTYPES[q.dtype],
            B, Hq, self.Hkv, self.seq_len, _ptr(seq_lens), ctypes.byref(kv), ctypes.byref(vv), float(scale),
            out.data_ptr(), _ptr(scores), self.workspace.data_ptr(), self.ws_bytes, _stream(stream)))
        return out

    def append_step(self, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, k_tail: PackedCache,
                    v_tail: PackedCache, kcache: PackedCache, vcache: PackedCache, scale: Optional[float] = None,
                    seq_lens: Optional[torch.Tensor] = None, scores: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """tq_append_decode_attention: encode the new token's K and V
        ([B, Hkv, d] or [B, Hkv, 1, d], same dtype) into the tail records
        k_tail / v_tail ([B, Hkv, 1] views, usually the last token of
        kcache / vcache), then attend over kcache / vcache."""
        B, Hq, d = q.shape
        assert (B, Hq) == (self.B, self.Hq) and q.is_contiguous() and q.dtype in _DTYPES
        if k_new.dim() == 4:
            k_new, v_new = k_new[:, :, 0], v_new[:, :, 0]
        assert k_new.shape == (B, self.Hkv, d) and v_new.shape == k_new.shape
        assert k_new.dtype == v_new.dtype and k_new.dtype in _DTYPES
        assert k_new.stride() == v_new.stride() and k_new.stride(2) == 1
        if scale is None:
            scale = 1.0 / math.sqrt(d)
        out = self.out if out is None else out
        kv, vv, kt, vt = kcache.view(), vcache.view(), k_tail.view(), v_tail.view()
        if seq_lens is not None:
            assert seq_lens.dtype == torch.int32 and seq_lens.is_contiguous()
        L.check(L.lib().tq_append_decode_attention(
            ctypes.byref(self.kq.c_struct()), ctypes.byref(self.vq.c_struct()), k_new.data_ptr(), v_new.data_ptr(),
            _DTYPES[k_new.dtype], k_new.stride(0), k_new.stride(1), ctypes.byref(kt), ctypes.byref(vt),
            q.data_ptr(), _DTYPES[q.dtype], B, Hq, self.Hkv, self.seq_len, _ptr(seq_lens), ctypes.byref(kv),
            ctypes.byref(vv), float(scale), out.data_ptr(), _ptr(scores), self.workspace.data_ptr(), self.ws_bytes,
            _stream(stream)))
        return out


def decode_attention(kq: Quantizer, vq: Quantizer, q: torch.Tensor, kcache: PackedCache, vcache: PackedCache,
                     scale: Optional[float] = None, seq_lens: Optional[torch.Tensor] = None,
                     scores: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One-shot tq_decode_attention (allocates its workspace and output)."""
    B, Hq, _ = q.shape
    _, Hkv, N = kcache.shape
    op = DecodeAttention(kq, vq, B, Hq, Hkv, N, device=q.device)
    return op(q, kcache, vcache, scale=scale, seq_lens=seq_lens, scores=scores).clone()


class SplitQuantizer:
    """Outlier-channel split of a d-channel head: group 0 (the outlier
    channels, ascending) at bits_o, group 1 (the rest) at bits_r, each its
    own dense-rotation quantizer reading its channels of the head."""

    def __init__(self, d: int, channels, bits_o: int, bits_r: int, variant: str = "mse", seed_rot: int = 0,
                 seed_qjl: int = 1, device="cuda"):
        ch = torch.as_tensor(channels, dtype=torch.int64).sort().values
        mask = torch.ones(d, dtype=torch.bool)
        mask[ch] = False
        rest = torch.nonzero(mask)[:, 0]
        self.d, self.channels, self.rest = d, ch, rest
        self.groups = (
            Quantizer(ch.numel(), bits_o, variant, seed_rot=seed_rot, seed_qjl=seed_qjl, device=device,
                      rotation="dense", channels=ch),
            Quantizer(rest.numel(), bits_r, variant, seed_rot=seed_rot + 1, seed_qjl=seed_qjl + 1, device=device,
                      rotation="dense", channels=rest))

    def c_array(self):
        return (L.TqQuantizer * 2)(self.groups[0].c_struct(), self.groups[1].c_struct())


def encode_split(sq: SplitQuantizer, x: torch.Tensor, stream=None):
    """tq_encode of both channel groups of x ([B, H, N, d] or fewer dims):
    (cache of group 0, cache of group 1)."""
    return tuple(encode(g, x, stream=stream) for g in sq.groups)


class DecodeAttentionSplit:
    """tq_decode_attention_split with its workspace allocated once."""

    def __init__(self, kq: SplitQuantizer, vq: SplitQuantizer, B: int, Hq: int, Hkv: int, seq_len: int,
                 device="cuda"):
        self.kq, self.vq, self.B, self.Hq, self.Hkv, self.seq_len = kq, vq, B, Hq, Hkv, seq_len
        nb = int(L.lib().tq_decode_split_workspace_bytes(B, Hq, Hkv, seq_len, kq.d))
        self.workspace = torch.empty(max(nb, 16), dtype=torch.uint8, device=device)
        self.ws_bytes = nb
        self.out = torch.empty((B, Hq, kq.d), dtype=torch.float32, device=device)

    def __call__(self, q: torch.Tensor, kcaches, vcaches, scale: Optional[float] = None,
                 seq_lens: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        B, Hq, d = q.shape
        assert (B, Hq, d) == (self.B, self.Hq, self.kq.d) and q.is_contiguous() and q.dtype in _DTYPES
        if scale is None:
            scale = 1.0 / math.sqrt(d)
        kv = (L.TqCacheView * 2)(kcaches[0].view(), kcaches[1].view())
        vv = (L.TqCacheView * 2)(vcaches[0].view(), vcaches[1].view())
        ka, va = self.kq.c_array(), self.vq.c_array()
        L.check(L.lib().tq_decode_attention_split(
            ka, va, q.data_ptr(), _DTYPES[q.dtype], B, Hq, self.Hkv, self.seq_len, _ptr(seq_lens), kv, vv,
            float(scale), self.out.data_ptr(), self.workspace.data_ptr(), self.ws_bytes, _stream(stream)))
        return self.out


class Search:
    """Reusable tq_search_topk call over a packed database of n_db records
    (its workspace allocated once)."""

    def __init__(self, qz: Quantizer, n_q: int, n_db: int, device="cuda"):
        self.qz, self.n_q, self.n_db = qz, n_q, n_db
        nb = int(L.lib().tq_search_workspace_bytes(n_q, n_db, qz.d))
        self.workspace = torch.empty(max(nb, 16), dtype=torch.uint8, device=device)
        self.ws_bytes = nb

    def __call__(self, queries: torch.Tensor, db: PackedCache, k: int, stream=None):
        """(top scores [n_q, k] fp32, top indices [n_q, k] int64) of the
        queries [n_q, d] against the n_db records of db (shaped [1, 1, n_db]
        or [n_db], any record stride)."""
        n_q, d = queries.shape
        assert n_q == self.n_q and d == self.qz.d and queries.is_contiguous() and queries.dtype in _DTYPES
        dev = queries.device
        top_v = _empty((n_q, k), torch.float32, dev, stream)
        top_i = _empty((n_q, k), torch.int64, dev, stream)
        v = db.view()
        L.check(L.lib().tq_search_topk(ctypes.byref(self.qz.c_struct()), ctypes.byref(v), self.n_db,
                                       queries.data_ptr(), _DTYPES[queries.dtype], n_q, k, top_v.data_ptr(),
                                       top_i.data_ptr(), self.workspace.data_ptr(), self.ws_bytes,
                                       _stream(stream)))
        return top_v, top_i


def search_topk(qz: Quantizer, queries: torch.Tensor, db: PackedCache, k: int):
    """One-shot tq_search_topk (allocates its workspace and outputs)."""
    n_db = db.norms.numel()
    return Search(qz, queries.shape[0], n_db, device=queries.device)(queries, db, k)


# ------------------------------------------------------------ paged cache

def _call(device: int, stream, fn, *args) -> None:
    """fn(*args, stream) with `device` current, on `stream` or that device's
    current one."""
    assert device >= 0, "the tensors of a paged call are on a CUDA device"
    s = _raw_stream(device) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() == device:
        status = fn(*args, s)
    else:
        with torch.cuda.device(device):
            status = fn(*args, s)
    if status != L.TQ_OK:
        L.check(status)


def _strides(t: Optional[torch.Tensor]):
    """Element strides over the first two dims (0 where the extent is 1)."""
    if t is None:
        return 0, 0
    (n, m, _), (a, b, c) = t.shape, t.stride()
    assert c == 1, "the last dim must be contiguous"
    return (a if n > 1 else 0), (b if m > 1 else 0)


def _check(device: int, dtype, **ts) -> None:
    """Contiguous tensors of one type on this device (None: not given)."""
    for name, t in ts.items():
        if t is not None and not (t.dtype is dtype and t.get_device() == device and t.is_contiguous()):
            raise AssertionError(f"{name}: a contiguous {dtype} tensor on device {device}, got {t.dtype} on {t.device}")


def _check_cache(device: int, qz: Quantizer, cache: PackedCache, shape) -> None:
    """A cache of this quantizer's records, norms of this shape, on this
    device: the kernels take the records' size from the quantizer alone."""
    codes, norms = cache.codes, cache.norms
    assert norms.dtype is torch.float32 and codes is not None and codes.dtype is torch.uint8, \
        "a cache has fp32 norms and uint8 codes"
    assert codes.shape == (*shape, qz.code_bytes), \
        f"codes {tuple(codes.shape)} are not those of {tuple(shape)} records of this quantizer"
    assert norms.get_device() == device and codes.get_device() == device and qz.signs.get_device() == device, \
        f"caches and quantizers must be on device {device}"


def _check_table(device: int, table: torch.Tensor, R: int):
    """(row stride, entries a row) of a block table [R, max_pages]."""
    (n, width), (stride, one) = table.shape, table.stride()
    assert n == R and table.dtype is torch.int32 and table.get_device() == device and (one == 1 or width <= 1), \
        "block_table: an int32 tensor [R, max_pages] on the call's device"
    return (stride if R > 1 else width), width


@dataclass
class PagePlan:
    """Outputs of tq_page_plan (views of the planner's buffers, overwritten
    by its next call)."""
    slots: torch.Tensor      # [max_tokens] int64, -1 where there is none
    positions: torch.Tensor  # [max_tokens] int32
    cu_new: torch.Tensor     # [R + 1] int32
    seq_lens: torch.Tensor   # [R] int32, new tokens included
    status: torch.Tensor     # [R] int32: 0, or why a request was refused
    n_free: torch.Tensor     # [1] int32, free pages left


class PagePlanner:
    """Reusable tq_page_plan call for n_requests requests and at most
    max_tokens new token rows (its outputs allocated once)."""

    def __init__(self, n_requests: int, page_size: int, max_tokens: int, device="cuda"):
        self.R, self.page_size, self.max_tokens = n_requests, page_size, max_tokens
        i32 = dict(dtype=torch.int32, device=device)
        self.plan = PagePlan(torch.empty(max_tokens, dtype=torch.int64, device=device), torch.empty(max_tokens, **i32),
                             torch.empty(n_requests + 1, **i32), torch.empty(n_requests, **i32),
                             torch.empty(n_requests, **i32), torch.empty(1, **i32))
        p = self.plan
        self.device = p.slots.get_device()
        self._out = tuple(t.data_ptr() for t in (p.slots, p.positions, p.cu_new, p.seq_lens, p.status, p.n_free))

    def __call__(self, lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor, n_free: torch.Tensor,
                 block_table: torch.Tensor, stream=None) -> PagePlan:
        """Give the new_lens [R] tokens that requests of lens [R] cached ones
        add their slots; new pages come off the end of free_pages[:n_free]
        (n_free: a one-element int32 device tensor) and are entered in
        block_table [R, max_pages] (int32, in place).  Pass plan.seq_lens and
        plan.n_free on by copying them: they may not be this call's inputs."""
        p, R = self.plan, self.R
        assert lens.shape == (R,) and new_lens.shape == (R,) and n_free.numel() == 1 and free_pages.dim() == 1
        _check(self.device, torch.int32, lens=lens, new_lens=new_lens, free_pages=free_pages, n_free=n_free)
        stride, width = _check_table(self.device, block_table, R)
        _call(self.device, stream, L.lib().tq_page_plan, R, self.page_size, lens.data_ptr(), new_lens.data_ptr(),
              free_pages.data_ptr(), free_pages.shape[0], n_free.data_ptr(), block_table.data_ptr(), stride, width,
              self.max_tokens, *self._out)
        return p


class Rope:
    """Rotary positions on several axes (tq_rope): inv_freq [rot_dim / 2]
    (fp32, on the device), and which axis turns which frequency, either as
    sections (how many consecutive frequencies each axis has) or as axis
    [rot_dim / 2] itself; neither means one axis.  pairing "half" turns the
    coordinates (f, f + rot_dim/2), "adjacent" (2f, 2f + 1)."""

    def __init__(self, inv_freq: torch.Tensor, sections=None, axis=None, pairing: str = "half"):
        assert pairing in ("half", "adjacent") and inv_freq.dim() == 1
        assert sections is None or axis is None
        self.inv_freq = inv_freq.to(torch.float32).contiguous()
        n = self.inv_freq.numel()
        if sections is not None:
            assert sum(sections) == n and all(c >= 0 for c in sections), "sections must cover the frequencies"
            axis = [a for a, c in enumerate(sections) for _ in range(c)]
            self.n_axes = len(sections)
        elif axis is not None:
            axis = [int(a) for a in axis]
            assert len(axis) == n and all(a >= 0 for a in axis)
            self.n_axes = max(axis) + 1
        else:
            self.n_axes = 1
        self.axis = None if axis is None else torch.tensor(axis, dtype=torch.int32).to(inv_freq.device)
        self.pairing, self.rot_dim = pairing, 2 * n
        self._c = L.TqRope(2 * n, L.TQ_ROPE_ADJACENT if pairing == "adjacent" else L.TQ_ROPE_HALF, self.n_axes,
                           _ptr(self.inv_freq), _ptr(self.axis))

        self._ref = ctypes.byref(self._c)

    def c_ref(self):
        return self._ref


def paged_append(kq: Quantizer, vq: Quantizer, k: torch.Tensor, v: torch.Tensor, kcache: PackedCache,
                 vcache: PackedCache, slots: torch.Tensor, q: Optional[torch.Tensor] = None,
                 rope: Optional[Rope] = None, positions: Optional[torch.Tensor] = None,
                 q_out: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """tq_paged_append: encode k and v [T, Hkv, d] into the records at
    slots [T] (int64; -1 skips a row) of kcache and vcache (empty_cache(qz,
    n_pages, Hkv, page_size)).  With a rope, k and the query rows q [T, Hq, d]
    are turned to positions ([T] or [n_axes, T], int32) first, and the turned
    q is returned (q_out, or a new tensor)."""
    T, Hkv, d = k.shape
    dev, dt = k.get_device(), k.dtype
    assert d == kq.d and v.shape == k.shape and v.dtype is dt and dt in _DTYPES
    assert v.get_device() == dev and slots.shape == (T,)
    _check(dev, torch.int64, slots=slots)
    n_pages, H, P = shape = kcache.norms.shape
    assert H == Hkv and vcache.norms.shape == shape
    _check_cache(dev, kq, kcache, shape)
    _check_cache(dev, vq, vcache, shape)
    pos_stride, rp, pp = 0, None, None
    if rope is not None:
        assert positions is not None and positions.dtype is torch.int32 and positions.get_device() == dev
        assert positions.shape == (rope.n_axes, T) or (rope.n_axes == 1 and positions.shape == (T,))
        assert T <= 1 or positions.stride(-1) == 1
        assert rope.inv_freq.get_device() == dev
        pos_stride = positions.stride(0) if rope.n_axes > 1 else 0
        rp, pp = rope.c_ref(), positions.data_ptr()
    else:
        assert q is None and positions is None, "query rows and positions need a rope"
    Hq = 0
    if q is not None:
        Hq = q.shape[1]
        assert q.shape == (T, Hq, d) and q.dtype is dt and q.get_device() == dev
        if q_out is None:
            q_out = _empty((T, Hq, d), dt, q.device, stream)
        assert q_out.shape == q.shape
        _check(dev, dt, q_out=q_out)
    _call(dev, stream, L.lib().tq_paged_append, kq.c_ref(), vq.c_ref(), rp, pp, pos_stride, _DTYPES[dt], T, Hq, Hkv,
          _ptr(q), *_strides(q), k.data_ptr(), *_strides(k), v.data_ptr(), *_strides(v), _ptr(q_out) if Hq else None,
          kcache.c_ref(), vcache.c_ref(), n_pages, P, slots.data_ptr())
    return q_out if q is not None else None


def paged_dequant(qz: Quantizer, cache: PackedCache, slots: torch.Tensor, dtype=torch.float32,
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """tq_paged_dequant: the vectors of the records at slots [T] (int64; -1
    gives zeros) as [T, H, d] in dtype."""
    n_pages, H, P = shape = cache.norms.shape
    (T,), dev = slots.shape, cache.norms.get_device()
    _check(dev, torch.int64, slots=slots)
    _check_cache(dev, qz, cache, shape)
    if out is None:
        out = _empty((T, H, qz.d), dtype, cache.norms.device, stream)
    assert out.shape == (T, H, qz.d) and out.dtype in _DTYPES
    _check(dev, out.dtype, out=out)
    _call(dev, stream, L.lib().tq_paged_dequant, qz.c_ref(), cache.c_ref(), n_pages, P, T, H, slots.data_ptr(),
          _DTYPES[out.dtype], out.data_ptr())
    return out


class PagedAttention:
    """Reusable tq_paged_attention call for batches of at most max_requests
    requests and max_tokens query rows (its workspace allocated once).  Calls
    that may overlap on the GPU need an object each, which is kept until they
    have run."""

    def __init__(self, kq: Quantizer, vq: Quantizer, Hq: int, Hkv: int, max_requests: int, max_tokens: int,
                 device="cuda"):
        self.kq, self.vq, self.Hq, self.Hkv = kq, vq, Hq, Hkv
        self.max_requests, self.max_tokens = max_requests, max_tokens
        with torch.cuda.device(torch.device(device)):
            nb = int(L.lib().tq_paged_attention_workspace_bytes(max_requests, max_tokens, Hq, Hkv, kq.d))
        self.workspace = torch.empty(max(nb, 16), dtype=torch.uint8, device=device)
        self.device, self._ws, self.ws_bytes = self.workspace.get_device(), self.workspace.data_ptr(), nb

    def __call__(self, q: torch.Tensor, kcache: PackedCache, vcache: PackedCache, block_table: torch.Tensor,
                 kv_lens: torch.Tensor, cu_q: Optional[torch.Tensor] = None, max_q: Optional[int] = None,
                 scale: Optional[float] = None, causal: bool = True, window: int = 0,
                 out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
        """Attention of the query rows q [T, Hq, d] (bf16 or fp16): request r
        owns rows cu_q[r]:cu_q[r+1] (cu_q None: one row each), its cached
        tokens are the kv_lens[r] ones of the pages block_table[r] (its own
        rows' included).  max_q: an upper bound of the row counts, by which the
        kernel is chosen (default: 1 without cu_q, else T, which for a batch of
        many requests takes tiles of 128 or 256 rows for a few: give it).
        Returns out [T, Hq, d] in q's dtype; lse [T, Hq] (fp32), if given, gets
        the logarithm of the softmax's sums."""
        (T, Hq, d), (R,), dt, dev = q.shape, kv_lens.shape, q.dtype, self.device
        n_pages, Hkv, P = shape = kcache.norms.shape
        assert (Hq, Hkv, d) == (self.Hq, self.Hkv, self.kq.d) and vcache.norms.shape == shape
        assert dt in _DTYPES and q.get_device() == dev
        assert R <= self.max_requests and T <= self.max_tokens, "more requests or rows than the workspace is for"
        assert cu_q is None or cu_q.shape == (R + 1,)
        _check(dev, torch.int32, kv_lens=kv_lens, cu_q=cu_q)
        _check_cache(dev, self.kq, kcache, shape)
        _check_cache(dev, self.vq, vcache, shape)
        stride, width = _check_table(dev, block_table, R)
        if max_q is None:
            max_q = 1 if cu_q is None else max(T, 1)
        if scale is None:
            scale = 1.0 / math.sqrt(d)
        if out is None:
            out = _empty((T, Hq, d), dt, q.device, stream)
        else:
            assert out.shape == q.shape
            _check(dev, dt, out=out)
        if lse is not None:
            assert lse.shape == (T, Hq)
            _check(dev, torch.float32, lse=lse)
        _call(dev, stream, L.lib().tq_paged_attention, self.kq.c_ref(), self.vq.c_ref(), q.data_ptr(), _DTYPES[dt], T,
              Hq, Hkv, *_strides(q), kcache.c_ref(), vcache.c_ref(), n_pages, P, block_table.data_ptr(), stride, R,
              width, kv_lens.data_ptr(), _ptr(cu_q), max_q, scale, int(causal), window, out.data_ptr(), _ptr(lse),
              self._ws, self.ws_bytes)
        return out


def set_decode_feed(staged: bool) -> bool:
    """Feed of the tensor-core decode for this process: bulk-copy staging
    through shared memory (True) or straight into registers (False, the
    default). Returns whether staging was on before."""
    prev = L.lib().tq_set_decode_feed(L.TQ_FEED_BULK_STAGED if staged else L.TQ_FEED_REGISTERS)
    return prev == L.TQ_FEED_BULK_STAGED


def check(stream=None) -> None:
    L.check(L.lib().tq_check(_stream(stream)))

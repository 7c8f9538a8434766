"""Serving from a paged cache: the binding of the ``msa_paged_*`` calls.

A ``PagedShape`` names the sizes, a ``PagedCache`` holds the pools and the
batch description, a ``Rope`` the rotation; each keeps its C struct, so that a
decode step marshals only what changes. The calls are those of ``include/msa.h``:

* ``msa_paged_append(shape, cache, rope, K, V, k_idx, Q, q_idx, Q_out, q_idx_out, workspace, stream=None)``
* ``msa_paged_sparse_attn(shape, cache, Q, q_idx, block_idx, O, LSE, workspace, stream=None)``
* ``msa_paged_dense_attn(shape, cache, Q, O, LSE, workspace, stream=None)``

and ``paged_append``, ``paged_sparse_attn``, ``paged_dense_attn`` allocate the
outputs. Tensors live on one GPU; a call runs on that GPU, on its current
stream unless ``stream`` is given.
"""
from __future__ import annotations

import ctypes
import struct
from ctypes import addressof
from dataclasses import dataclass

from . import (MSA_ERR_UNSUPPORTED, MSA_WS_PAGED_APPEND, MSA_WS_PAGED_DENSE, MSA_WS_PAGED_SPARSE, MsaError, _check, _on_stream,
               load_library)


class MsaPagedShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("S", "N", "Hq", "G", "d", "d_idx", "Bk", "k", "num_pages", "max_blocks",
                                              "prefix_blocks")] + [("scale", ctypes.c_float)]


class MsaPagedCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("K", "V", "k_idx", "page_table", "row_start", "seq_len")]


class MsaRope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("inv_freq_idx", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("rot_dim_idx", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class MsaNewRows(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("Q", "K", "V", "q_idx", "k_idx")] + [
        (n, ctypes.c_int64) for n in ("ld_Q", "ld_K", "ld_V", "ld_q_idx", "ld_k_idx")]


@dataclass(frozen=True)
class PagedShape:
    S: int
    N: int
    Hq: int
    G: int
    num_pages: int
    max_blocks: int
    k: int = 16
    prefix_blocks: int = 0
    d: int = 128
    d_idx: int = 64
    Bk: int = 128
    scale: float = 0.0

    def __post_init__(self):
        # what every call would work out again: the C struct (not its address, which a copy does not share) and the
        # shapes of the tensors
        put = lambda n, v: object.__setattr__(self, n, v)  # noqa: E731
        put("_c", MsaPagedShape(self.S, self.N, self.Hq, self.G, self.d, self.d_idx, self.Bk, self.k, self.num_pages,
                                self.max_blocks, self.prefix_blocks, self.scale))
        put("_sizes", (self.S, self.G, self.num_pages, self.max_blocks, self.d, self.Bk))
        N, Hq, G = self.N, self.Hq, self.G
        put("_q", (N, Hq, self.d))
        put("_kv", (N, G, self.d))
        put("_qi", (N, G, self.d_idx))
        put("_ki", (N, self.d_idx))
        put("_bi", (N, G, self.k))
        put("_lse", (N, Hq))

    def c(self) -> MsaPagedShape:
        return self._c


_torch = _bf16 = None
_new_rows = struct.Struct("5P5q").pack  # the bytes of a MsaNewRows (in a sixth of the time)


def _t():
    """torch, imported at the first use (a PagedCache's, at the latest)."""
    global _torch, _bf16
    if _torch is None:
        import torch

        _torch, _bf16 = torch, torch.bfloat16
    return _torch


def _refuse(name, t, dtype, shape, device, packed=True):
    if not t.is_cuda and device != -1:
        raise ValueError(f"{name} must live on the GPU")
    if t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, {dtype} is needed")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, {tuple(shape)} is needed")
    if t.get_device() != device:
        raise ValueError(f"{name} lives on {t.device}, the cache on cuda:{device}")
    raise ValueError(f"{name} must be contiguous" if packed else f"the rows of {name} must be packed")


def _want(name, t, dtype, shape, device):
    """Address of a packed tensor of this type and shape on GPU `device`."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    _refuse(name, t, dtype, shape, device)


class _Fixed:
    """Has a C struct with its tensors' addresses: no tensor is replaced afterwards, and a copy has a struct of its own."""

    _held = ()  # the attributes in question

    def __setattr__(self, name, value):
        self._keep(name)
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        self._keep(name)
        object.__delattr__(self, name)

    def _keep(self, name):
        if name in self._held:
            raise AttributeError(f"{name} of a {type(self).__name__} cannot be replaced (the calls use the tensor's "
                                 f"address): write into the tensor, or make another {type(self).__name__}")

    def __reduce__(self):
        return type(self), self._args


class PagedCache(_Fixed):
    """Pools K, V [num_pages, G, 128, 128] and k_idx [num_pages, 128, 64] (or None) in bf16, and the batch description
    page_table [S, max_blocks], row_start [S + 1], seq_len [S] in int32. The tensors are kept as they are: their
    contents may change between calls, neither they nor their storage may be replaced."""

    _held = ("K", "V", "k_idx", "page_table", "row_start", "seq_len", "device")

    def __init__(self, K, V, k_idx, page_table, row_start, seq_len):
        torch = _t()
        if not K.is_cuda:
            raise ValueError("K must live on the GPU")
        pages, G, Bk, d = K.shape
        dev = K.get_device()
        S = seq_len.shape[0]
        bf, i32 = torch.bfloat16, torch.int32
        struct = MsaPagedCache(
            _want("K", K, bf, (pages, G, Bk, d), dev), _want("V", V, bf, (pages, G, Bk, d), dev),
            None if k_idx is None else _want("k_idx", k_idx, bf, (pages, Bk, k_idx.shape[-1]), dev),
            _want("page_table", page_table, i32, (S, page_table.shape[-1]), dev),
            _want("row_start", row_start, i32, (S + 1,), dev), _want("seq_len", seq_len, i32, (S,), dev))
        self.__dict__.update(
            K=K, V=V, k_idx=k_idx, page_table=page_table, row_start=row_start, seq_len=seq_len, device=K.device,
            _args=(K, V, k_idx, page_table, row_start, seq_len), _struct=struct, _addr=addressof(struct), _device=dev,
            _sizes=(S, G, pages, page_table.shape[-1], d, Bk), _index_dim=None if k_idx is None else k_idx.shape[-1])

    def check(self, shape):
        """The cache is one of `shape`."""
        if self._sizes != shape._sizes:
            raise ValueError(f"the cache has (S, G, num_pages, max_blocks, d, Bk) = {self._sizes}, the shape {shape._sizes}")
        if self._index_dim is not None and self._index_dim != shape.d_idx:
            raise ValueError(f"the cache's index keys have {self._index_dim} dims, the shape {shape.d_idx}")


class Rope(_Fixed):
    """Rotation frequencies (radians per position, fp32): inv_freq [rot_dim / 2] for Q and K, inv_freq_idx
    [rot_dim_idx / 2] for the index branch; None rotates nothing."""

    _held = ("inv_freq", "inv_freq_idx")

    def __init__(self, inv_freq=None, inv_freq_idx=None, interleaved=False):
        torch = _t()

        def ptr(name, t):
            if t is None or t.numel() == 0:
                return None, 0
            if not t.is_cuda:
                raise ValueError(f"{name} must live on the GPU")
            return _want(name, t, torch.float32, (t.numel(),), t.get_device()), 2 * t.numel()

        p, n = ptr("inv_freq", inv_freq)
        pi, ni = ptr("inv_freq_idx", inv_freq_idx)
        struct = MsaRope(p, pi, n, ni, 1 if interleaved else 0)
        self.__dict__.update(
            inv_freq=inv_freq, inv_freq_idx=inv_freq_idx, _args=(inv_freq, inv_freq_idx, interleaved), _struct=struct,
            _addr=addressof(struct),
            _devices={t.get_device() for t, q in ((inv_freq, p), (inv_freq_idx, pi)) if q is not None})


def _rows(name, t, shape, device):
    """Address and row stride of a [N, ...] input whose rows are packed (the pieces of a fused projection are)."""
    if t.dtype is not _bf16 or t.shape != shape or t.get_device() != device:
        _refuse(name, t, _bf16, shape, device, packed=False)
    if t.is_contiguous():
        return t.data_ptr(), 0
    strides, packed = t.stride(), 1
    if shape[0] > 1 and strides[-1] == 1 and (len(shape) == 2 or strides[1] == shape[2]):
        ld, packed = strides[0], shape[-1] if len(shape) == 2 else shape[1] * shape[2]
    else:
        for n, st in zip(shape[:0:-1], strides[:0:-1]):
            if n != 1 and st != packed:
                _refuse(name, t, t.dtype, shape, device, packed=False)
            packed *= n
        ld = strides[0] if shape[0] > 1 else packed
    if ld < packed:  # rows that lie on one another; expanded ones have stride 0, which the C call takes for packed rows
        raise ValueError(f"the rows of {name} must not overlap (their stride is {ld}): make an expanded tensor contiguous")
    return t.data_ptr(), ld


def _run(call, cache, stream, workspace, *args):
    """call(*args, workspace, its bytes, stream) with the cache's GPU current."""
    torch, dev = _torch, cache._device
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be contiguous on {cache.device}")
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    ws, n = workspace.data_ptr(), workspace.nbytes
    if torch._C._cuda_getDevice() == dev:
        status = call(*args, ws, n, stream)
    else:
        with torch.cuda.device(dev):
            status = call(*args, ws, n, stream)
    if status:
        _check(status)


def msa_paged_workspace_size(shape, which: int) -> int:
    return int(load_library().msa_paged_workspace_size(addressof(shape._c), which))


def alloc_paged_workspace(shape, which: int, device="cuda"):
    n = msa_paged_workspace_size(shape, which)
    if n == 0:
        raise MsaError(MSA_ERR_UNSUPPORTED, "shape not supported (see include/msa.h)")
    return _t().empty(n, dtype=_t().uint8, device=device)


def msa_paged_append(shape, cache, rope, K, V, k_idx, Q, q_idx, Q_out, q_idx_out, workspace, stream=None) -> None:
    """New tokens into their pages, K and k_idx rotated; Q and q_idx rotated into Q_out and q_idx_out. Inputs may be
    row-strided. k_idx, and Q or q_idx with its output, may be None."""
    cache.check(shape)
    dev = cache._device
    if k_idx is not None and cache.k_idx is None:
        raise ValueError("the cache has no index keys (k_idx)")
    if rope._devices and rope._devices != {dev}:
        raise ValueError(f"the rotation's frequencies must live on {cache.device}")
    none = (0, 0)
    kp, k_ld = _rows("K", K, shape._kv, dev)
    vp, v_ld = _rows("V", V, shape._kv, dev)
    qp, q_ld = none if Q is None else _rows("Q", Q, shape._q, dev)
    ip, i_ld = none if q_idx is None else _rows("q_idx", q_idx, shape._qi, dev)
    xp, x_ld = none if k_idx is None else _rows("k_idx", k_idx, shape._ki, dev)
    _run(load_library().msa_paged_append, cache, stream, workspace, addressof(shape._c), cache._addr, rope._addr,
         _new_rows(qp, kp, vp, ip, xp, q_ld, k_ld, v_ld, i_ld, x_ld),
         None if Q_out is None else _want("Q_out", Q_out, _bf16, shape._q, dev),
         None if q_idx_out is None else _want("q_idx_out", q_idx_out, _bf16, shape._qi, dev))


def msa_paged_sparse_attn(shape, cache, Q, q_idx, block_idx, O, LSE, workspace, stream=None) -> None:
    """Selection (q_idx given: block_idx is written; None: block_idx is read) and attention over the selected pages."""
    torch, bf = _torch, _bf16
    cache.check(shape)
    dev = cache._device
    if q_idx is not None and cache.k_idx is None:
        raise ValueError("the cache has no index keys (k_idx)")
    _run(load_library().msa_paged_sparse_attn, cache, stream, workspace, addressof(shape._c), cache._addr,
         _want("Q", Q, bf, shape._q, dev), None if q_idx is None else _want("q_idx", q_idx, bf, shape._qi, dev),
         _want("block_idx", block_idx, torch.int32, shape._bi, dev), _want("O", O, bf, shape._q, dev),
         _want("LSE", LSE, torch.float32, shape._lse, dev))


def msa_paged_dense_attn(shape, cache, Q, O, LSE, workspace, stream=None) -> None:
    """Full attention for the new rows; the first shape.prefix_blocks pages are those of every sequence."""
    torch, bf = _torch, _bf16
    cache.check(shape)
    dev = cache._device
    _run(load_library().msa_paged_dense_attn, cache, stream, workspace, addressof(shape._c), cache._addr,
         _want("Q", Q, bf, shape._q, dev), _want("O", O, bf, shape._q, dev),
         _want("LSE", LSE, torch.float32, shape._lse, dev))


# ----------------------------------------------------------------- allocation helpers
def paged_append(shape, cache, rope, K, V, k_idx=None, Q=None, q_idx=None, workspace=None, stream=None):
    """Allocate the rotated queries, run msa_paged_append and return (Q_out, q_idx_out); None where none was given."""
    dev = cache.device
    if stream is not None:
        return _on_stream(stream, dev, paged_append, shape, cache, rope, K, V, k_idx, Q, q_idx, workspace)
    ws = workspace if workspace is not None else alloc_paged_workspace(shape, MSA_WS_PAGED_APPEND, dev)
    Q_out = None if Q is None else _torch.empty(shape._q, dtype=_bf16, device=dev)
    qi_out = None if q_idx is None else _torch.empty(shape._qi, dtype=_bf16, device=dev)
    msa_paged_append(shape, cache, rope, K, V, k_idx, Q, q_idx, Q_out, qi_out, ws)
    return Q_out, qi_out


def paged_sparse_attn(shape, cache, Q, q_idx=None, block_idx=None, workspace=None, stream=None):
    """Allocate O, LSE (and block_idx, when q_idx selects) and run msa_paged_sparse_attn; returns (O, LSE, block_idx)."""
    dev = cache.device
    if stream is not None:
        return _on_stream(stream, dev, paged_sparse_attn, shape, cache, Q, q_idx, block_idx, workspace)
    if block_idx is None:
        if q_idx is None:
            raise ValueError("give q_idx to select blocks, or the block_idx to attend to")
        block_idx = _torch.empty(shape._bi, dtype=_torch.int32, device=dev)
    ws = workspace if workspace is not None else alloc_paged_workspace(shape, MSA_WS_PAGED_SPARSE, dev)
    O = _torch.empty(shape._q, dtype=_bf16, device=dev)
    LSE = _torch.empty(shape._lse, dtype=_torch.float32, device=dev)
    msa_paged_sparse_attn(shape, cache, Q, q_idx, block_idx, O, LSE, ws)
    return O, LSE, block_idx


def paged_dense_attn(shape, cache, Q, workspace=None, stream=None):
    """Allocate O and LSE and run msa_paged_dense_attn."""
    dev = cache.device
    if stream is not None:
        return _on_stream(stream, dev, paged_dense_attn, shape, cache, Q, workspace)
    ws = workspace if workspace is not None else alloc_paged_workspace(shape, MSA_WS_PAGED_DENSE, dev)
    O = _torch.empty(shape._q, dtype=_bf16, device=dev)
    LSE = _torch.empty(shape._lse, dtype=_torch.float32, device=dev)
    msa_paged_dense_attn(shape, cache, Q, O, LSE, ws)
    return O, LSE

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
from dataclasses import dataclass, field

from . import (MSA_ERR_UNSUPPORTED, MSA_WS_PAGED_APPEND, MSA_WS_PAGED_DENSE, MSA_WS_PAGED_SPARSE, MsaError, _check,
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
    _c: list = field(default_factory=list, init=False, repr=False, compare=False)

    def c(self) -> MsaPagedShape:
        if not self._c:
            self._c.append(MsaPagedShape(self.S, self.N, self.Hq, self.G, self.d, self.d_idx, self.Bk, self.k,
                                         self.num_pages, self.max_blocks, self.prefix_blocks, self.scale))
        return self._c[0]


def _want(name, t, dtype, shape=None, device=None):
    """A GPU tensor of this type and shape (None in the shape: any size), packed."""
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    if t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, {dtype} is needed")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, {tuple(shape)} is needed")
    if device is not None and t.device != device:
        raise ValueError(f"{name} lives on {t.device}, the cache on {device}")
    return t.data_ptr()


class PagedCache:
    """Pools K, V [num_pages, G, 128, 128] and k_idx [num_pages, 128, 64] (or None) in bf16, and the batch description
    page_table [S, max_blocks], row_start [S + 1], seq_len [S] in int32. The tensors are kept as they are; their
    contents may change between calls."""

    def __init__(self, K, V, k_idx, page_table, row_start, seq_len):
        import torch

        pages, G, Bk, d = K.shape
        dev = K.device
        S = seq_len.shape[0]
        bf, i32 = torch.bfloat16, torch.int32
        self._struct = MsaPagedCache(
            _want("K", K, bf), _want("V", V, bf, (pages, G, Bk, d), dev),
            None if k_idx is None else _want("k_idx", k_idx, bf, (pages, Bk, k_idx.shape[-1]), dev),
            _want("page_table", page_table, i32, (S, page_table.shape[-1]), dev),
            _want("row_start", row_start, i32, (S + 1,), dev), _want("seq_len", seq_len, i32, (S,), dev))
        self.K, self.V, self.k_idx = K, V, k_idx
        self.page_table, self.row_start, self.seq_len = page_table, row_start, seq_len
        self.device = dev
        self.sizes = (S, G, pages, page_table.shape[-1], d, Bk)
        self.index_dim = None if k_idx is None else k_idx.shape[-1]

    def check(self, shape):
        """The cache is one of `shape`."""
        if self.sizes != (shape.S, shape.G, shape.num_pages, shape.max_blocks, shape.d, shape.Bk):
            raise ValueError(f"the cache has (S, G, num_pages, max_blocks, d, Bk) = {self.sizes}, the shape "
                             f"{(shape.S, shape.G, shape.num_pages, shape.max_blocks, shape.d, shape.Bk)}")
        if self.index_dim is not None and self.index_dim != shape.d_idx:
            raise ValueError(f"the cache's index keys have {self.index_dim} dims, the shape {shape.d_idx}")


class Rope:
    """Rotation frequencies (radians per position, fp32): inv_freq [rot_dim / 2] for Q and K, inv_freq_idx
    [rot_dim_idx / 2] for the index branch; None rotates nothing."""

    def __init__(self, inv_freq=None, inv_freq_idx=None, interleaved=False):
        import torch

        def ptr(name, t):
            if t is None or t.numel() == 0:
                return None, 0
            return _want(name, t, torch.float32, (t.numel(),)), 2 * t.numel()

        p, n = ptr("inv_freq", inv_freq)
        pi, ni = ptr("inv_freq_idx", inv_freq_idx)
        self.inv_freq, self.inv_freq_idx = inv_freq, inv_freq_idx
        self.devices = [t.device for t in (inv_freq, inv_freq_idx) if t is not None]
        self._struct = MsaRope(p, pi, n, ni, 1 if interleaved else 0)


def _rows(name, t, shape, device):
    """Address and row stride of a [N, ...] input whose rows are packed (the pieces of a fused projection are)."""
    import torch

    if t.dtype != torch.bfloat16 or t.device != device:
        raise ValueError(f"{name} must be bfloat16 on {device}, it is {t.dtype} on {t.device}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, {shape} is needed")
    packed = 1
    for n, st in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if n != 1 and st != packed:
            raise ValueError(f"the rows of {name} must be packed")
        packed *= n
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else packed


def _call(cache, stream, workspace, run):
    """run(workspace, its bytes, stream) with the cache's GPU current."""
    import torch

    if workspace.device != cache.device or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be contiguous on {cache.device}")
    dev = cache.device.index
    here = torch.cuda.current_device()
    if dev != here:
        torch.cuda.set_device(dev)
    try:
        if stream is None:
            stream = torch.cuda.current_stream(dev)
        raw = stream if isinstance(stream, int) else stream.cuda_stream
        _check(run(workspace.data_ptr(), workspace.numel() * workspace.element_size(), raw))
    finally:
        if dev != here:
            torch.cuda.set_device(here)


def msa_paged_workspace_size(shape, which: int) -> int:
    return int(load_library().msa_paged_workspace_size(ctypes.addressof(shape.c()), which))


def alloc_paged_workspace(shape, which: int, device="cuda"):
    import torch

    n = msa_paged_workspace_size(shape, which)
    if n == 0:
        raise MsaError(MSA_ERR_UNSUPPORTED, "shape not supported (see include/msa.h)")
    return torch.empty(n, dtype=torch.uint8, device=device)


def msa_paged_append(shape, cache, rope, K, V, k_idx, Q, q_idx, Q_out, q_idx_out, workspace, stream=None) -> None:
    """New tokens into their pages, K and k_idx rotated; Q and q_idx rotated into Q_out and q_idx_out. Inputs may be
    row-strided. k_idx, and Q or q_idx with its output, may be None."""
    import torch

    cache.check(shape)
    N, dev = shape.N, cache.device
    if k_idx is not None and cache.k_idx is None:
        raise ValueError("the cache has no index keys (k_idx)")
    if any(d != dev for d in rope.devices):
        raise ValueError(f"the rotation's frequencies must live on {dev}")
    r = MsaNewRows()
    r.K, r.ld_K = _rows("K", K, (N, shape.G, shape.d), dev)
    r.V, r.ld_V = _rows("V", V, (N, shape.G, shape.d), dev)
    out = qi_out = None
    if Q is not None:
        r.Q, r.ld_Q = _rows("Q", Q, (N, shape.Hq, shape.d), dev)
    if q_idx is not None:
        r.q_idx, r.ld_q_idx = _rows("q_idx", q_idx, (N, shape.G, shape.d_idx), dev)
    if k_idx is not None:
        r.k_idx, r.ld_k_idx = _rows("k_idx", k_idx, (N, shape.d_idx), dev)
    if Q_out is not None:
        out = _want("Q_out", Q_out, torch.bfloat16, (N, shape.Hq, shape.d), dev)
    if q_idx_out is not None:
        qi_out = _want("q_idx_out", q_idx_out, torch.bfloat16, (N, shape.G, shape.d_idx), dev)
    lib = load_library()
    _call(cache, stream, workspace, lambda ws, n, st: lib.msa_paged_append(
        ctypes.addressof(shape.c()), ctypes.addressof(cache._struct), ctypes.addressof(rope._struct),
        ctypes.addressof(r), out, qi_out, ws, n, st))


def msa_paged_sparse_attn(shape, cache, Q, q_idx, block_idx, O, LSE, workspace, stream=None) -> None:
    """Selection (q_idx given: block_idx is written; None: block_idx is read) and attention over the selected pages."""
    import torch

    cache.check(shape)
    N, dev, bf = shape.N, cache.device, torch.bfloat16
    if q_idx is not None and cache.k_idx is None:
        raise ValueError("the cache has no index keys (k_idx)")
    args = (_want("Q", Q, bf, (N, shape.Hq, shape.d), dev),
            None if q_idx is None else _want("q_idx", q_idx, bf, (N, shape.G, shape.d_idx), dev),
            _want("block_idx", block_idx, torch.int32, (N, shape.G, shape.k), dev),
            _want("O", O, bf, (N, shape.Hq, shape.d), dev), _want("LSE", LSE, torch.float32, (N, shape.Hq), dev))
    lib = load_library()
    _call(cache, stream, workspace, lambda ws, n, st: lib.msa_paged_sparse_attn(
        ctypes.addressof(shape.c()), ctypes.addressof(cache._struct), *args, ws, n, st))


def msa_paged_dense_attn(shape, cache, Q, O, LSE, workspace, stream=None) -> None:
    """Full attention for the new rows; the first shape.prefix_blocks pages are those of every sequence."""
    import torch

    cache.check(shape)
    N, dev, bf = shape.N, cache.device, torch.bfloat16
    args = (_want("Q", Q, bf, (N, shape.Hq, shape.d), dev), _want("O", O, bf, (N, shape.Hq, shape.d), dev),
            _want("LSE", LSE, torch.float32, (N, shape.Hq), dev))
    lib = load_library()
    _call(cache, stream, workspace, lambda ws, n, st: lib.msa_paged_dense_attn(
        ctypes.addressof(shape.c()), ctypes.addressof(cache._struct), *args, ws, n, st))


# ----------------------------------------------------------------- allocation helpers
def paged_append(shape, cache, rope, K, V, k_idx=None, Q=None, q_idx=None, workspace=None, stream=None):
    """Allocate the rotated queries, run msa_paged_append and return (Q_out, q_idx_out); None where none was given."""
    import torch

    dev = cache.device
    ws = workspace if workspace is not None else alloc_paged_workspace(shape, MSA_WS_PAGED_APPEND, dev)
    Q_out = None if Q is None else torch.empty((shape.N, shape.Hq, shape.d), dtype=torch.bfloat16, device=dev)
    qi_out = None if q_idx is None else torch.empty((shape.N, shape.G, shape.d_idx), dtype=torch.bfloat16, device=dev)
    msa_paged_append(shape, cache, rope, K, V, k_idx, Q, q_idx, Q_out, qi_out, ws, stream)
    return Q_out, qi_out


def paged_sparse_attn(shape, cache, Q, q_idx=None, block_idx=None, workspace=None, stream=None):
    """Allocate O, LSE (and block_idx, when q_idx selects) and run msa_paged_sparse_attn; returns (O, LSE, block_idx)."""
    import torch

    dev = cache.device
    ws = workspace if workspace is not None else alloc_paged_workspace(shape, MSA_WS_PAGED_SPARSE, dev)
    if block_idx is None:
        if q_idx is None:
            raise ValueError("give q_idx to select blocks, or the block_idx to attend to")
        block_idx = torch.empty((shape.N, shape.G, shape.k), dtype=torch.int32, device=dev)
    O = torch.empty((shape.N, shape.Hq, shape.d), dtype=torch.bfloat16, device=dev)
    LSE = torch.empty((shape.N, shape.Hq), dtype=torch.float32, device=dev)
    msa_paged_sparse_attn(shape, cache, Q, q_idx, block_idx, O, LSE, ws, stream)
    return O, LSE, block_idx


def paged_dense_attn(shape, cache, Q, workspace=None, stream=None):
    """Allocate O and LSE and run msa_paged_dense_attn."""
    import torch

    dev = cache.device
    ws = workspace if workspace is not None else alloc_paged_workspace(shape, MSA_WS_PAGED_DENSE, dev)
    O = torch.empty((shape.N, shape.Hq, shape.d), dtype=torch.bfloat16, device=dev)
    LSE = torch.empty((shape.N, shape.Hq), dtype=torch.float32, device=dev)
    msa_paged_dense_attn(shape, cache, Q, O, LSE, ws, stream)
    return O, LSE

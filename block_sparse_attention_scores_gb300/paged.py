"""Serving from a paged cache: the binding of the ``msa_paged_*`` calls.

A ``PagedShape`` names the sizes, a ``PagedCache`` holds the pools and the
batch description, a ``Rope`` the rotation; each keeps its C struct, so that a
decode step marshals only what changes. The calls are those of ``include/msa.h``:

* ``msa_paged_append(shape, cache, rope, K, V, k_idx, Q, q_idx, Q_out, q_idx_out, workspace, stream=None, positions=None)``
* ``msa_paged_sparse_attn(shape, cache, Q, q_idx, block_idx, O, LSE, workspace, stream=None)``
* ``msa_paged_dense_attn(shape, cache, Q, O, LSE, workspace, stream=None)``

and ``paged_append``, ``paged_sparse_attn``, ``paged_dense_attn`` allocate the
outputs. The same calls with ``_fp8`` at their end take a ``PagedCacheFp8``, which
holds E4M3 codes and powers of two, and ``msa_paged_read_fp8`` (``paged_read_fp8``)
gives its tokens back as bf16. Tensors live on one GPU; a call runs on that GPU, on its current
stream unless ``stream`` is given.
"""
from __future__ import annotations

import ctypes
import struct
from ctypes import addressof
from dataclasses import dataclass

from . import (MSA_ERR_UNSUPPORTED, MSA_WS_PAGED_APPEND, MSA_WS_PAGED_DENSE, MSA_WS_PAGED_DENSE_FP8, MSA_WS_PAGED_SPARSE,
               MSA_WS_PAGED_SPARSE_FP8, MsaError, _check, _on_stream, load_library)


class MsaPagedShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("S", "N", "Hq", "G", "d", "d_idx", "Bk", "k", "num_pages", "max_blocks",
                                              "prefix_blocks")] + [("scale", ctypes.c_float)]


class MsaPagedCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("K", "V", "k_idx", "page_table", "row_start", "seq_len")]


class MsaPagedCacheFp8(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("K", "V", "K_exp", "V_exp", "k_idx", "k_idx_exp", "page_table", "row_start",
                                               "seq_len")]


class MsaAxes(ctypes.Structure):
    _fields_ = [("positions", ctypes.c_void_p), ("axis", ctypes.c_void_p), ("axis_idx", ctypes.c_void_p),
                ("axes", ctypes.c_int32)]


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
_axes = struct.Struct("3Pi4x").pack     # and of a MsaAxes


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


class _Cache(_Fixed):
    def check(self, shape):
        """The cache is one of `shape`."""
        if self._sizes != shape._sizes:
            raise ValueError(f"the cache has (S, G, num_pages, max_blocks, d, Bk) = {self._sizes}, the shape {shape._sizes}")
        if self._index_dim is not None and self._index_dim != shape.d_idx:
            raise ValueError(f"the cache's index keys have {self._index_dim} dims, the shape {shape.d_idx}")

    def _hold(self, args, struct, **tensors):
        K, table = tensors["K"], tensors["page_table"]
        pages, G, Bk, d = K.shape
        k_idx = tensors["k_idx"]
        self.__dict__.update(
            tensors, device=K.device, _args=args, _struct=struct, _addr=addressof(struct), _device=K.get_device(),
            _sizes=(tensors["seq_len"].shape[0], G, pages, table.shape[-1], d, Bk),
            _index_dim=None if k_idx is None else k_idx.shape[-1])


class PagedCache(_Cache):
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
        self._hold((K, V, k_idx, page_table, row_start, seq_len), struct, K=K, V=V, k_idx=k_idx, page_table=page_table,
                   row_start=row_start, seq_len=seq_len)


class PagedCacheFp8(_Cache):
    """A cache in 8 bits: pools K, V [num_pages, G, 128, 128] and k_idx [num_pages, 128, 64] (or None) in
    torch.float8_e4m3fn, and the exponents + 127 of their vectors' powers of two, K_exp, V_exp [num_pages, G, 128] and
    k_idx_exp [num_pages, 128] in uint8; the batch description as a PagedCache's. The tensors are kept as they are."""

    _held = ("K", "V", "K_exp", "V_exp", "k_idx", "k_idx_exp", "page_table", "row_start", "seq_len", "device")

    def __init__(self, K, V, K_exp, V_exp, k_idx, k_idx_exp, page_table, row_start, seq_len):
        torch = _t()
        if not K.is_cuda:
            raise ValueError("K must live on the GPU")
        if (k_idx is None) != (k_idx_exp is None):
            raise ValueError("give k_idx with k_idx_exp, or neither")
        pages, G, Bk, d = K.shape
        dev = K.get_device()
        S = seq_len.shape[0]
        f8, u8, i32 = torch.float8_e4m3fn, torch.uint8, torch.int32
        struct = MsaPagedCacheFp8(
            _want("K", K, f8, (pages, G, Bk, d), dev), _want("V", V, f8, (pages, G, Bk, d), dev),
            _want("K_exp", K_exp, u8, (pages, G, Bk), dev), _want("V_exp", V_exp, u8, (pages, G, Bk), dev),
            None if k_idx is None else _want("k_idx", k_idx, f8, (pages, Bk, k_idx.shape[-1]), dev),
            None if k_idx is None else _want("k_idx_exp", k_idx_exp, u8, (pages, Bk), dev),
            _want("page_table", page_table, i32, (S, page_table.shape[-1]), dev),
            _want("row_start", row_start, i32, (S + 1,), dev), _want("seq_len", seq_len, i32, (S,), dev))
        self._hold((K, V, K_exp, V_exp, k_idx, k_idx_exp, page_table, row_start, seq_len), struct, K=K, V=V, K_exp=K_exp,
                   V_exp=V_exp, k_idx=k_idx, k_idx_exp=k_idx_exp, page_table=page_table, row_start=row_start,
                   seq_len=seq_len)


class Rope(_Fixed):
    """Rotation frequencies (radians per position, fp32): inv_freq [rot_dim / 2] for Q and K, inv_freq_idx
    [rot_dim_idx / 2] for the index branch; None rotates nothing. For positions with several axes, axis and axis_idx
    (int32, as long) name each pair's axis; None: all on axis 0."""

    _held = ("inv_freq", "inv_freq_idx", "axis", "axis_idx")

    def __init__(self, inv_freq=None, inv_freq_idx=None, interleaved=False, axis=None, axis_idx=None):
        torch = _t()

        def ptr(name, t, kind, length=None):
            if t is None or t.numel() == 0:
                return None, 0
            if not t.is_cuda:
                raise ValueError(f"{name} must live on the GPU")
            return _want(name, t, kind, (t.numel() if length is None else length,), t.get_device()), 2 * t.numel()

        p, n = ptr("inv_freq", inv_freq, torch.float32)
        pi, ni = ptr("inv_freq_idx", inv_freq_idx, torch.float32)
        ax, _ = ptr("axis", axis, torch.int32, n // 2)
        axi, _ = ptr("axis_idx", axis_idx, torch.int32, ni // 2)
        struct = MsaRope(p, pi, n, ni, 1 if interleaved else 0)
        given = ((inv_freq, p), (inv_freq_idx, pi), (axis, ax), (axis_idx, axi))
        self.__dict__.update(
            inv_freq=inv_freq, inv_freq_idx=inv_freq_idx, axis=axis, axis_idx=axis_idx,
            _args=(inv_freq, inv_freq_idx, interleaved, axis, axis_idx), _struct=struct, _addr=addressof(struct),
            _axis=ax, _axis_idx=axi, _devices={t.get_device() for t, q in given if q is not None})


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


def _is(kind, cache):
    """The cache is of the type that the call takes."""
    if type(cache) is not kind and not isinstance(cache, kind):
        raise TypeError(f"a {kind.__name__} is needed, not a {type(cache).__name__}")


def _append(kind, shape, cache, rope, K, V, k_idx, Q, q_idx, Q_out, q_idx_out, workspace, stream, positions):
    _is(kind, cache)
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
    lib, axes = load_library(), None
    if positions is not None:
        n = positions.shape[-1] if positions.dim() == 2 else 0
        axes = _axes(_want("positions", positions, _torch.int32, (shape.N, n), dev), rope._axis or 0, rope._axis_idx or 0, n)
    elif rope._axis or rope._axis_idx:
        raise ValueError("the rotation has axes: give the rows' positions on them")
    rows = _new_rows(qp, kp, vp, ip, xp, q_ld, k_ld, v_ld, i_ld, x_ld)
    out = (None if Q_out is None else _want("Q_out", Q_out, _bf16, shape._q, dev),
           None if q_idx_out is None else _want("q_idx_out", q_idx_out, _bf16, shape._qi, dev))
    if kind is PagedCacheFp8:
        _run(lib.msa_paged_append_fp8, cache, stream, workspace, addressof(shape._c), cache._addr, rope._addr, axes, rows, *out)
    elif axes is None:
        _run(lib.msa_paged_append, cache, stream, workspace, addressof(shape._c), cache._addr, rope._addr, rows, *out)
    else:
        _run(lib.msa_paged_append_axes, cache, stream, workspace, addressof(shape._c), cache._addr, rope._addr, axes, rows, *out)


def _sparse(kind, call, shape, cache, Q, q_idx, block_idx, O, LSE, workspace, stream):
    _is(kind, cache)
    torch, bf = _torch, _bf16
    cache.check(shape)
    dev = cache._device
    if q_idx is not None and cache.k_idx is None:
        raise ValueError("the cache has no index keys (k_idx)")
    _run(call, cache, stream, workspace, addressof(shape._c), cache._addr,
         _want("Q", Q, bf, shape._q, dev), None if q_idx is None else _want("q_idx", q_idx, bf, shape._qi, dev),
         _want("block_idx", block_idx, torch.int32, shape._bi, dev), _want("O", O, bf, shape._q, dev),
         _want("LSE", LSE, torch.float32, shape._lse, dev))


def _dense(kind, call, shape, cache, Q, O, LSE, workspace, stream):
    _is(kind, cache)
    torch, bf = _torch, _bf16
    cache.check(shape)
    dev = cache._device
    _run(call, cache, stream, workspace, addressof(shape._c), cache._addr,
         _want("Q", Q, bf, shape._q, dev), _want("O", O, bf, shape._q, dev),
         _want("LSE", LSE, torch.float32, shape._lse, dev))


def msa_paged_append(shape, cache, rope, K, V, k_idx, Q, q_idx, Q_out, q_idx_out, workspace, stream=None,
                     positions=None) -> None:
    """New tokens into their pages, K and k_idx rotated; Q and q_idx rotated into Q_out and q_idx_out. Inputs may be
    row-strided. k_idx, and Q or q_idx with its output, may be None. positions [N, axes] (int32): the rows' positions on
    the axes that the rotation's pairs turn on; None: in their sequences."""
    _append(PagedCache, shape, cache, rope, K, V, k_idx, Q, q_idx, Q_out, q_idx_out, workspace, stream, positions)


def msa_paged_append_fp8(shape, cache, rope, K, V, k_idx, Q, q_idx, Q_out, q_idx_out, workspace, stream=None,
                         positions=None) -> None:
    """msa_paged_append into a PagedCacheFp8: K, V and k_idx are quantised as they are written."""
    _append(PagedCacheFp8, shape, cache, rope, K, V, k_idx, Q, q_idx, Q_out, q_idx_out, workspace, stream, positions)


def msa_paged_sparse_attn(shape, cache, Q, q_idx, block_idx, O, LSE, workspace, stream=None) -> None:
    """Selection (q_idx given: block_idx is written; None: block_idx is read) and attention over the selected pages."""
    _sparse(PagedCache, load_library().msa_paged_sparse_attn, shape, cache, Q, q_idx, block_idx, O, LSE, workspace, stream)


def msa_paged_sparse_attn_fp8(shape, cache, Q, q_idx, block_idx, O, LSE, workspace, stream=None) -> None:
    """msa_paged_sparse_attn over a PagedCacheFp8."""
    _sparse(PagedCacheFp8, load_library().msa_paged_sparse_attn_fp8, shape, cache, Q, q_idx, block_idx, O, LSE, workspace,
            stream)


def msa_paged_dense_attn(shape, cache, Q, O, LSE, workspace, stream=None) -> None:
    """Full attention for the new rows; the first shape.prefix_blocks pages are those of every sequence."""
    _dense(PagedCache, load_library().msa_paged_dense_attn, shape, cache, Q, O, LSE, workspace, stream)


def msa_paged_dense_attn_fp8(shape, cache, Q, O, LSE, workspace, stream=None) -> None:
    """msa_paged_dense_attn over a PagedCacheFp8."""
    _dense(PagedCacheFp8, load_library().msa_paged_dense_attn_fp8, shape, cache, Q, O, LSE, workspace, stream)


def msa_paged_read_fp8(shape, cache, first, out_start, K_out, V_out, k_idx_out, workspace, stream=None) -> None:
    """Tokens of a PagedCacheFp8 as bf16: rows out_start[s] .. out_start[s + 1] - 1 of K_out, V_out [M, G, 128] and
    k_idx_out [M, 64] (or None) are the tokens from first[s] on of sequence s (first None: from its beginning).
    first [S] and out_start [S + 1] are int32; rows before out_start[0] and from out_start[S] on are left alone."""
    _is(PagedCacheFp8, cache)
    cache.check(shape)
    dev, i32, M = cache._device, _torch.int32, K_out.shape[0]
    if k_idx_out is not None and cache.k_idx is None:
        raise ValueError("the cache has no index keys (k_idx)")
    _run(load_library().msa_paged_read_fp8, cache, stream, workspace, addressof(shape._c), cache._addr,
         None if first is None else _want("first", first, i32, (shape.S,), dev),
         _want("out_start", out_start, i32, (shape.S + 1,), dev), M,
         _want("K_out", K_out, _bf16, (M, shape.G, shape.d), dev), _want("V_out", V_out, _bf16, (M, shape.G, shape.d), dev),
         None if k_idx_out is None else _want("k_idx_out", k_idx_out, _bf16, (M, shape.d_idx), dev))


# ----------------------------------------------------------------- allocation helpers
def _new_append(call, shape, cache, rope, K, V, k_idx, Q, q_idx, workspace, positions):
    dev = cache.device
    ws = workspace if workspace is not None else alloc_paged_workspace(shape, MSA_WS_PAGED_APPEND, dev)
    Q_out = None if Q is None else _torch.empty(shape._q, dtype=_bf16, device=dev)
    qi_out = None if q_idx is None else _torch.empty(shape._qi, dtype=_bf16, device=dev)
    call(shape, cache, rope, K, V, k_idx, Q, q_idx, Q_out, qi_out, ws, positions=positions)
    return Q_out, qi_out


def _new_sparse(call, which, shape, cache, Q, q_idx, block_idx, workspace):
    dev = cache.device
    if block_idx is None:
        if q_idx is None:
            raise ValueError("give q_idx to select blocks, or the block_idx to attend to")
        block_idx = _torch.empty(shape._bi, dtype=_torch.int32, device=dev)
    ws = workspace if workspace is not None else alloc_paged_workspace(shape, which, dev)
    O = _torch.empty(shape._q, dtype=_bf16, device=dev)
    LSE = _torch.empty(shape._lse, dtype=_torch.float32, device=dev)
    call(shape, cache, Q, q_idx, block_idx, O, LSE, ws)
    return O, LSE, block_idx


def _new_dense(call, which, shape, cache, Q, workspace):
    dev = cache.device
    ws = workspace if workspace is not None else alloc_paged_workspace(shape, which, dev)
    O = _torch.empty(shape._q, dtype=_bf16, device=dev)
    LSE = _torch.empty(shape._lse, dtype=_torch.float32, device=dev)
    call(shape, cache, Q, O, LSE, ws)
    return O, LSE


def paged_append(shape, cache, rope, K, V, k_idx=None, Q=None, q_idx=None, workspace=None, stream=None, positions=None):
    """Allocate the rotated queries, run msa_paged_append and return (Q_out, q_idx_out); None where none was given."""
    args = msa_paged_append, shape, cache, rope, K, V, k_idx, Q, q_idx, workspace, positions
    return _new_append(*args) if stream is None else _on_stream(stream, cache.device, _new_append, *args)


def paged_append_fp8(shape, cache, rope, K, V, k_idx=None, Q=None, q_idx=None, workspace=None, stream=None, positions=None):
    """paged_append for a PagedCacheFp8."""
    args = msa_paged_append_fp8, shape, cache, rope, K, V, k_idx, Q, q_idx, workspace, positions
    return _new_append(*args) if stream is None else _on_stream(stream, cache.device, _new_append, *args)


def paged_sparse_attn(shape, cache, Q, q_idx=None, block_idx=None, workspace=None, stream=None):
    """Allocate O, LSE (and block_idx, when q_idx selects) and run msa_paged_sparse_attn; returns (O, LSE, block_idx)."""
    args = msa_paged_sparse_attn, MSA_WS_PAGED_SPARSE, shape, cache, Q, q_idx, block_idx, workspace
    return _new_sparse(*args) if stream is None else _on_stream(stream, cache.device, _new_sparse, *args)


def paged_sparse_attn_fp8(shape, cache, Q, q_idx=None, block_idx=None, workspace=None, stream=None):
    """paged_sparse_attn over a PagedCacheFp8."""
    args = msa_paged_sparse_attn_fp8, MSA_WS_PAGED_SPARSE_FP8, shape, cache, Q, q_idx, block_idx, workspace
    return _new_sparse(*args) if stream is None else _on_stream(stream, cache.device, _new_sparse, *args)


def paged_dense_attn(shape, cache, Q, workspace=None, stream=None):
    """Allocate O and LSE and run msa_paged_dense_attn."""
    args = msa_paged_dense_attn, MSA_WS_PAGED_DENSE, shape, cache, Q, workspace
    return _new_dense(*args) if stream is None else _on_stream(stream, cache.device, _new_dense, *args)


def paged_dense_attn_fp8(shape, cache, Q, workspace=None, stream=None):
    """paged_dense_attn over a PagedCacheFp8."""
    args = msa_paged_dense_attn_fp8, MSA_WS_PAGED_DENSE_FP8, shape, cache, Q, workspace
    return _new_dense(*args) if stream is None else _on_stream(stream, cache.device, _new_dense, *args)


def _new_read(shape, cache, out_start, M, first, workspace):
    dev = cache.device
    ws = workspace if workspace is not None else alloc_paged_workspace(shape, MSA_WS_PAGED_APPEND, dev)
    K, V = (_torch.empty((M, shape.G, shape.d), dtype=_bf16, device=dev) for _ in range(2))
    k_idx = None if cache.k_idx is None else _torch.empty((M, shape.d_idx), dtype=_bf16, device=dev)
    msa_paged_read_fp8(shape, cache, first, out_start, K, V, k_idx, ws)
    return K, V, k_idx


def paged_read_fp8(shape, cache, out_start, M, first=None, workspace=None, stream=None):
    """Allocate K, V [M, G, 128] and k_idx [M, 64] (None without index keys), run msa_paged_read_fp8 and return them."""
    args = shape, cache, out_start, M, first, workspace
    return _new_read(*args) if stream is None else _on_stream(stream, cache.device, _new_read, *args)

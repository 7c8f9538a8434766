"""The paged-cache calls check their arguments before any device work (no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__

    __graft_entry__.build_library()
    import block_sparse_attention_scores_gb300 as m

    return m


BASE = dict(S=2, N=3, Hq=8, G=2, num_pages=10, max_blocks=4, k=4)
P = 4096  # an aligned address that is never followed: every case here is refused on the host


def _shape(msa, **kw):
    return msa.PagedShape(**{**BASE, **kw})


def _cache(msa, **kw):
    from block_sparse_attention_scores_gb300.paged import MsaPagedCache

    return MsaPagedCache(**{**dict(K=P, V=P, k_idx=P, page_table=P, row_start=P, seq_len=P), **kw})


def _rope(msa, **kw):
    from block_sparse_attention_scores_gb300.paged import MsaRope

    return MsaRope(**{**dict(inv_freq=P, inv_freq_idx=P, rot_dim=128, rot_dim_idx=64, interleaved=0), **kw})


def _rows(msa, **kw):
    from block_sparse_attention_scores_gb300.paged import MsaNewRows

    return MsaNewRows(**{**dict(Q=P, K=P, V=P, q_idx=P, k_idx=P), **kw})


def _status(msa, f):
    with pytest.raises(msa.MsaError) as e:
        msa._check(f())
    return e.value.status, str(e.value)


def _append(msa, shape=None, cache=None, rope=None, rows=None, Q_out=P, q_idx_out=P, ws=P, n=1 << 40):
    lib, a = msa.load_library(), ctypes.addressof
    shape, cache = shape or _shape(msa).c(), cache or _cache(msa)
    rope, rows = rope or _rope(msa), rows or _rows(msa)
    return _status(msa, lambda: lib.msa_paged_append(a(shape), a(cache), a(rope), a(rows), Q_out, q_idx_out, ws, n, 0))


def _sparse(msa, shape=None, cache=None, Q=P, q_idx=P, block_idx=P, O=P, LSE=P, ws=P, n=1 << 40):
    lib, a = msa.load_library(), ctypes.addressof
    shape, cache = shape or _shape(msa).c(), cache or _cache(msa)
    return _status(msa, lambda: lib.msa_paged_sparse_attn(a(shape), a(cache), Q, q_idx, block_idx, O, LSE, ws, n, 0))


def _dense(msa, shape=None, cache=None, Q=P, O=P, LSE=P, ws=P, n=1 << 40):
    lib, a = msa.load_library(), ctypes.addressof
    shape, cache = shape or _shape(msa).c(), cache or _cache(msa)
    return _status(msa, lambda: lib.msa_paged_dense_attn(a(shape), a(cache), Q, O, LSE, ws, n, 0))


@pytest.mark.parametrize("kw,status", [
    (dict(S=0), "INVALID_ARG"), (dict(N=0), "INVALID_ARG"), (dict(Hq=0), "INVALID_ARG"), (dict(G=0), "INVALID_ARG"),
    (dict(k=0), "INVALID_ARG"), (dict(num_pages=0), "INVALID_ARG"), (dict(max_blocks=0), "INVALID_ARG"),
    (dict(prefix_blocks=-1), "INVALID_ARG"), (dict(prefix_blocks=4), "INVALID_ARG"), (dict(Hq=7), "INVALID_ARG"),
    (dict(scale=float("inf")), "INVALID_ARG"), (dict(d=64), "UNSUPPORTED"), (dict(d_idx=32), "UNSUPPORTED"),
    (dict(Bk=64), "UNSUPPORTED"), (dict(Hq=32), "UNSUPPORTED"), (dict(Hq=6), "UNSUPPORTED"),
    (dict(k=129), "UNSUPPORTED"), (dict(S=65536), "UNSUPPORTED"), (dict(max_blocks=8193), "UNSUPPORTED"),
    (dict(N=(1 << 20) + 1), "UNSUPPORTED"), (dict(num_pages=1 << 23), "UNSUPPORTED"),
    (dict(N=1 << 20, Hq=1024, G=128), "UNSUPPORTED"),
])
def test_shapes_outside_the_contract(msa, kw, status):
    s = _shape(msa, **kw)
    want = getattr(msa, "MSA_ERR_" + status)
    for which in (msa.MSA_WS_PAGED_APPEND, msa.MSA_WS_PAGED_SPARSE, msa.MSA_WS_PAGED_DENSE):
        assert msa.msa_paged_workspace_size(s, which) == 0
    assert _append(msa, shape=s.c())[0] == want
    assert _sparse(msa, shape=s.c())[0] == want
    assert _dense(msa, shape=s.c())[0] == want


def test_workspace_sizes(msa):
    s = _shape(msa)
    sizes = [msa.msa_paged_workspace_size(s, w) for w in range(3)]
    assert sizes[0] == 256 and sizes[1] > 256 and sizes[2] > 256
    assert msa.msa_paged_workspace_size(s, 3) == 0 and msa.msa_paged_workspace_size(s, -1) == 0
    # the prefix belongs to the dense call alone
    p = _shape(msa, prefix_blocks=3)
    assert msa.msa_paged_workspace_size(p, msa.MSA_WS_PAGED_SPARSE) == sizes[1]
    # the scores of every row and block
    big = _shape(msa, N=64, max_blocks=8192, num_pages=1 << 20, G=8, Hq=32)
    assert msa.msa_paged_workspace_size(big, msa.MSA_WS_PAGED_SPARSE) > 64 * 8 * 8192 * 4


@pytest.mark.parametrize("name", ["K", "V", "page_table", "row_start", "seq_len"])
def test_cache_pointers(msa, name):
    for bad, what in ((None, "NULL"), (P + 2, "aligned")):
        c = _cache(msa, **{name: bad})
        for call in (_append, _sparse, _dense):
            st, msg = call(msa, cache=c)
            assert st == msa.MSA_ERR_INVALID_ARG and name in msg and what in msg


def test_index_keys_are_needed_with_an_index_branch_only(msa):
    c = _cache(msa, k_idx=None)
    assert "k_idx" in _sparse(msa, cache=c)[1]
    assert "k_idx" in _append(msa, cache=c)[1]
    assert _sparse(msa, cache=c, q_idx=None, ws=None)[0] == msa.MSA_ERR_WORKSPACE  # past the pointer checks
    assert _append(msa, cache=c, rows=_rows(msa, k_idx=None), ws=None)[0] == msa.MSA_ERR_WORKSPACE


@pytest.mark.parametrize("name", ["Q", "block_idx", "O", "LSE"])
def test_sparse_pointers(msa, name):
    st, msg = _sparse(msa, **{name: None})
    assert st == msa.MSA_ERR_INVALID_ARG and name in msg
    st, msg = _sparse(msa, **{name: P + 1})
    assert st == msa.MSA_ERR_INVALID_ARG and "aligned" in msg
    if name != "block_idx":
        assert name in _dense(msa, **{name: None})[1]


def test_append_arguments(msa):
    inv = msa.MSA_ERR_INVALID_ARG
    for name in ("K", "V"):
        st, msg = _append(msa, rows=_rows(msa, **{name: None}))
        assert st == inv and name in msg
    for name in ("Q", "K", "V", "q_idx", "k_idx"):
        assert "aligned" in _append(msa, rows=_rows(msa, **{name: P + 8}))[1]
        for ld in (8, 2052, -2048):  # shorter than a row, not a multiple of 16 bytes, negative
            if name == "k_idx" and ld == 8:
                ld = 56
            st, msg = _append(msa, rows=_rows(msa, **{"ld_" + name: ld}))
            assert st == inv and "stride of " + name in msg
    # an input and its output come together
    assert "Q_out" in _append(msa, Q_out=None)[1]
    assert "Q_out" in _append(msa, rows=_rows(msa, Q=None))[1]
    assert "q_idx_out" in _append(msa, q_idx_out=None)[1]
    assert "q_idx_out" in _append(msa, rows=_rows(msa, q_idx=None))[1]
    for kw in (dict(rot_dim=144), dict(rot_dim=-16), dict(rot_dim=24), dict(rot_dim_idx=80), dict(rot_dim_idx=8)):
        st, msg = _append(msa, rope=_rope(msa, **kw))
        assert st == inv and "rot_dim" in msg
    assert "inv_freq " in _append(msa, rope=_rope(msa, inv_freq=None))[1]
    assert "inv_freq_idx" in _append(msa, rope=_rope(msa, inv_freq_idx=None))[1]
    # no index vectors: their rotation is not looked at
    r = _rows(msa, q_idx=None, k_idx=None)
    assert _append(msa, rope=_rope(msa, inv_freq_idx=None, rot_dim_idx=8), rows=r, q_idx_out=None, ws=None)[0] == \
        msa.MSA_ERR_WORKSPACE


def test_null_structs(msa):
    lib, a = msa.load_library(), ctypes.addressof
    s, c, r, n = _shape(msa).c(), _cache(msa), _rope(msa), _rows(msa)
    for args in ((None, a(c), a(r), a(n)), (a(s), None, a(r), a(n)), (a(s), a(c), None, a(n)), (a(s), a(c), a(r), None)):
        assert _status(msa, lambda: lib.msa_paged_append(*args, P, P, P, 1 << 20, 0))[0] == msa.MSA_ERR_INVALID_ARG
    assert _status(msa, lambda: lib.msa_paged_sparse_attn(a(s), None, P, P, P, P, P, P, 1 << 20, 0))[0] == \
        msa.MSA_ERR_INVALID_ARG
    assert _status(msa, lambda: lib.msa_paged_dense_attn(None, a(c), P, P, P, P, 1 << 20, 0))[0] == \
        msa.MSA_ERR_INVALID_ARG


def test_workspace_is_checked(msa):
    for call in (_append, _sparse, _dense):
        assert call(msa, ws=None)[0] == msa.MSA_ERR_WORKSPACE
        assert "aligned" in call(msa, ws=P + 128)[1]
        st, msg = call(msa, n=255)
        assert st == msa.MSA_ERR_WORKSPACE and "needed" in msg


def test_binding_refuses_tensors_of_another_kind(msa):
    import torch

    from block_sparse_attention_scores_gb300.paged import _rows as rows

    with pytest.raises(ValueError, match="GPU"):
        msa.PagedCache(*[torch.zeros(2, 2, 128, 128, dtype=torch.bfloat16)] * 2, None,
                       torch.zeros(2, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32),
                       torch.zeros(2, dtype=torch.int32))
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    assert rows("K", x, (3, 2, 128), -1)[1] == 0  # packed
    fused = torch.zeros(3, 640, dtype=torch.bfloat16)[:, 128:384].unflatten(1, (2, 128))
    assert rows("K", fused, (3, 2, 128), -1)[1] == 640
    with pytest.raises(ValueError, match="packed"):
        rows("K", torch.zeros(2, 3, 128, dtype=torch.bfloat16).transpose(0, 1), (3, 2, 128), -1)[1] and rows(
            "K", torch.zeros(3, 128, 2, dtype=torch.bfloat16).transpose(1, 2), (3, 2, 128), -1)
    with pytest.raises(ValueError, match="shape"):
        rows("K", x, (3, 4, 128), -1)
    with pytest.raises(ValueError, match="bfloat16"):
        rows("K", x.float(), (3, 2, 128), -1)


@pytest.mark.parametrize("x,shape", [
    ((1, 2, 128), (64, 2, 128)), ((1, 1, 128), (64, 1, 128)), ((1, 64), (64, 64)), ((1, 1, 64), (9, 2, 64)),
    ((3, 1, 128), (3, 2, 128)), ((1, 1, 1), (3, 2, 128)),
], ids=str)
def test_binding_refuses_expanded_rows(msa, x, shape):
    """A row stride of 0 means packed rows to the C call, which would read past the end of an expanded tensor."""
    import torch

    from block_sparse_attention_scores_gb300.paged import _rows as rows

    t = torch.zeros(x, dtype=torch.bfloat16).expand(shape)
    with pytest.raises(ValueError, match="overlap|packed"):
        rows("K", t, shape, -1)
    assert rows("K", t.contiguous(), shape, -1)[1] == 0


def test_binding_refuses_overlapping_rows(msa):
    import torch

    from block_sparse_attention_scores_gb300.paged import _rows as rows

    for ld in (0, 8, 128, 248):
        t = torch.zeros(1024, dtype=torch.bfloat16).as_strided((3, 2, 128), (ld, 128, 1))
        with pytest.raises(ValueError, match="overlap"):
            rows("K", t, (3, 2, 128), -1)
    # one group: the stride between groups says nothing
    t = torch.zeros(1024, dtype=torch.bfloat16).as_strided((3, 1, 128), (0, 640, 1))
    with pytest.raises(ValueError, match="overlap"):
        rows("K", t, (3, 1, 128), -1)
    # a single row may have any stride
    t = torch.zeros(1024, dtype=torch.bfloat16).as_strided((1, 2, 128), (0, 128, 1))
    assert rows("K", t, (1, 2, 128), -1)[1] in (0, 256)
    assert rows("k_idx", torch.zeros(1, 64, dtype=torch.bfloat16).expand(1, 64), (1, 64), -1)[1] in (0, 64)


@pytest.mark.parametrize("how", ["copy", "deepcopy", "pickle", "replace"])
def test_copied_shapes_stand_on_their_own(msa, how):
    """A copy works after its original is gone, and in another process: it holds no address of the original's struct."""
    import copy
    import dataclasses
    import gc
    import pickle

    kw = dict(N=7, max_blocks=40, num_pages=100)
    want = [msa.msa_paged_workspace_size(_shape(msa, **kw), w) for w in range(3)]
    s = _shape(msa, **kw)
    assert not [n for n, v in vars(s).items() if isinstance(v, int) and n.startswith("_")]
    c = {"copy": copy.copy, "deepcopy": copy.deepcopy, "pickle": lambda x: pickle.loads(pickle.dumps(x)),
         "replace": dataclasses.replace}[how](s)
    del s
    gc.collect()
    others = [_shape(msa, N=1 + i) for i in range(50)]  # what takes its memory
    assert len(others) == 50
    assert [msa.msa_paged_workspace_size(c, w) for w in range(3)] == want
    assert c == _shape(msa, **kw)


def test_pickled_shape_in_another_process(msa):
    import pathlib
    import pickle
    import subprocess
    import sys

    s = _shape(msa, N=7, max_blocks=40, num_pages=100)
    code = ("import pickle, sys\n"
            "import block_sparse_attention_scores_gb300 as msa\n"
            "s = pickle.loads(bytes.fromhex(sys.argv[1]))\n"
            "print(msa.msa_paged_workspace_size(s, msa.MSA_WS_PAGED_DENSE))\n")
    out = subprocess.run([sys.executable, "-c", code, pickle.dumps(s).hex()], capture_output=True, text=True, timeout=600,
                         cwd=pathlib.Path(__file__).resolve().parent.parent)
    assert out.returncode == 0, out.stderr[-2000:]
    assert int(out.stdout) == msa.msa_paged_workspace_size(s, msa.MSA_WS_PAGED_DENSE)


@pytest.mark.parametrize("kind,names", [("PagedCache", ("K", "V", "k_idx", "page_table", "row_start", "seq_len")),
                                        ("Rope", ("inv_freq", "inv_freq_idx"))])
def test_tensors_of_a_cache_are_not_replaced(msa, kind, names):
    """The calls go by the addresses taken when the object was made: a replaced tensor would be a freed one to them."""
    import copy
    import pickle

    rope = msa.Rope(interleaved=True)
    thing = rope if kind == "Rope" else msa.PagedCache.__new__(msa.PagedCache)
    for n in names:
        with pytest.raises(AttributeError, match=f"{n} of a {kind}"):
            setattr(thing, n, None)
        with pytest.raises(AttributeError, match=f"{n} of a {kind}"):
            delattr(thing, n)
    thing.layer = 3  # a user's own
    for c in (copy.copy(rope), copy.deepcopy(rope), pickle.loads(pickle.dumps(rope))):
        assert c._addr == ctypes.addressof(c._struct) != rope._addr
        assert (c._struct.rot_dim, c._struct.rot_dim_idx, c._struct.interleaved) == (0, 0, 1)


def _slots(msa, shape):
    """Parts of a row's output that the full call's workspace has room for."""
    return msa.msa_paged_workspace_size(shape, msa.MSA_WS_PAGED_DENSE) // (shape.N * shape.Hq * 516)


@pytest.mark.parametrize("kw", [dict(S=1, N=128, Hq=64, G=8, prefix_blocks=187), dict(S=2, N=64, Hq=64, G=8, prefix_blocks=60),
                                dict(S=1, N=127, Hq=32, G=8, prefix_blocks=50), dict(S=4, N=128, Hq=64, G=8, prefix_blocks=40),
                                dict(S=60000, N=160, Hq=8, G=1, prefix_blocks=9)],  # nearly all of them idle
                         ids=str)
def test_a_prefix_that_many_rows_read_is_shared(msa, kw):
    """A prefix is read as own pages where that is little work: its pages count once for every tile of eight columns, not
    once for every sequence (one sequence's 128 rows would read theirs 128 times)."""
    shape = msa.PagedShape(**kw, num_pages=1000, max_blocks=kw["prefix_blocks"] + 1)
    # (one part of the own page, and the prefix cut into more than one; read as own pages it is not cut at all)
    assert _slots(msa, shape) >= 3


@pytest.mark.parametrize("Hq,G", [(65544, 65544), (1 << 17, 1 << 17), (1 << 23, 1 << 20), (1 << 27, 1 << 24)], ids=str)
def test_more_heads_than_are_counted(msa, Hq, G):
    """A row of more than 2^22 16-byte pieces would lose its last ones, and pages times groups leave 32 bits."""
    s = _shape(msa, N=1, S=1, Hq=Hq, G=G, num_pages=1, max_blocks=8192)
    for which in range(3):
        assert msa.msa_paged_workspace_size(s, which) == 0
    for call in (_append, _sparse, _dense):
        st, msg = call(msa, shape=s.c())
        assert st == msa.MSA_ERR_UNSUPPORTED and ("Hq" in msg or "G" in msg)
    s = _shape(msa, N=1, S=1, Hq=65536, G=65536, num_pages=1, max_blocks=8)
    assert msa.msa_paged_workspace_size(s, msa.MSA_WS_PAGED_DENSE) > 0


def test_workspaces_hold_what_is_written(msa):
    """No parts of outputs where rows are not cut, no block maxima where nothing is chosen between blocks."""
    def sparse(**kw):
        base = dict(S=1, N=32768, Hq=64, G=8, num_pages=1000, max_blocks=256, k=16)
        return msa.msa_paged_workspace_size(msa.PagedShape(**{**base, **kw}), msa.MSA_WS_PAGED_SPARSE)

    rows = 32768 * (32 + 8 * 12)          # their places, and counters
    pooled = 32768 * 8 * 256 * 8          # a block's maximum and its keys' largest value
    assert rows + pooled <= sparse() < rows + pooled + 4096
    assert rows <= sparse(k=1) < rows + 4096
    assert sparse(max_blocks=1) < rows + 4096
    dense = msa.msa_paged_workspace_size(msa.PagedShape(S=32768, N=32768, Hq=64, G=8, num_pages=1000, max_blocks=2),
                                         msa.MSA_WS_PAGED_DENSE)
    assert rows <= dense < rows + 4096
    # few rows are cut: as many parts as before
    one = msa.msa_paged_workspace_size(msa.PagedShape(S=1, N=1, Hq=32, G=8, num_pages=1000, max_blocks=100),
                                       msa.MSA_WS_PAGED_DENSE)
    assert one > 2 * 32 * 516


def test_a_shared_prefix_leaves_sms_to_the_own_pages(msa):
    """64 sequences behind 256 pages with 16 pages of their own: the prefix's runs take half of the SMs (93 us; 108 with
    nearly all of them), so a row has few parts of it."""
    kw = dict(N=64, Hq=32, G=8, num_pages=5000, max_blocks=272, prefix_blocks=256)
    few, all_of = _slots(msa, msa.PagedShape(S=64, **kw)), 152 * 256 / (8 * 256)
    assert few - 1 <= 0.6 * all_of

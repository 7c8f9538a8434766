"""The calls over a paged cache in 8 bits, and positions with several axes: arguments are checked before any device work
(no GPU needed); the test reference's format against torch's conversions."""
import ctypes

import pytest

import paged_fp8_ref as ref8


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__

    __graft_entry__.build_library()
    import block_sparse_attention_scores_gb300 as m

    return m


BASE = dict(S=2, N=3, Hq=8, G=2, num_pages=10, max_blocks=4, k=4)
P = 4096  # an aligned address that is never followed: every case here is refused on the host
POOLS = ("K", "V", "K_exp", "V_exp", "k_idx", "k_idx_exp")


def _shape(msa, **kw):
    return msa.PagedShape(**{**BASE, **kw})


def _struct(name, **kw):
    from block_sparse_attention_scores_gb300 import paged

    kind = getattr(paged, name)
    base = {n: P for n, t in kind._fields_ if t is ctypes.c_void_p}
    base.update(dict(MsaRope=dict(rot_dim=128, rot_dim_idx=64), MsaAxes=dict(axes=3)).get(name, {}))
    return kind(**{**base, **kw})


def _call(msa, name, args, ws=P, n=1 << 40):
    with pytest.raises(msa.MsaError) as e:
        msa._check(getattr(msa.load_library(), name)(*[ctypes.addressof(x) if isinstance(x, ctypes.Structure) else x
                                                       for x in args], ws, n, 0))
    return e.value.status, str(e.value)


def _append(msa, shape=None, cache=None, rope=None, axes=P, rows=None, Q_out=P, q_idx_out=P, bf16=False, **kw):
    axes = _struct("MsaAxes") if axes == P else axes
    cache = cache or _struct("MsaPagedCache" if bf16 else "MsaPagedCacheFp8")
    return _call(msa, "msa_paged_append_axes" if bf16 else "msa_paged_append_fp8",
                 (shape or _shape(msa).c(), cache, rope or _struct("MsaRope"), axes, rows or _struct("MsaNewRows"), Q_out,
                  q_idx_out), **kw)


def _read(msa, shape=None, cache=None, first=P, out_start=P, M=5, K=P, V=P, k_idx=P, **kw):
    return _call(msa, "msa_paged_read_fp8", (shape or _shape(msa).c(), cache or _struct("MsaPagedCacheFp8"), first, out_start,
                                             M, K, V, k_idx), **kw)


def _sparse(msa, shape=None, cache=None, Q=P, q_idx=P, block_idx=P, O=P, LSE=P, **kw):
    return _call(msa, "msa_paged_sparse_attn_fp8", (shape or _shape(msa).c(), cache or _struct("MsaPagedCacheFp8"), Q, q_idx,
                                                    block_idx, O, LSE), **kw)


def _dense(msa, shape=None, cache=None, Q=P, O=P, LSE=P, **kw):
    return _call(msa, "msa_paged_dense_attn_fp8", (shape or _shape(msa).c(), cache or _struct("MsaPagedCacheFp8"), Q, O, LSE),
                 **kw)


CALLS = (_append, _read, _sparse, _dense)


@pytest.mark.parametrize("kw,status", [
    (dict(S=0), "INVALID_ARG"), (dict(N=0), "INVALID_ARG"), (dict(Hq=7), "INVALID_ARG"), (dict(k=0), "INVALID_ARG"),
    (dict(prefix_blocks=4), "INVALID_ARG"), (dict(scale=float("inf")), "INVALID_ARG"), (dict(d=64), "UNSUPPORTED"),
    (dict(d_idx=32), "UNSUPPORTED"), (dict(Bk=64), "UNSUPPORTED"), (dict(Hq=32), "UNSUPPORTED"), (dict(k=129), "UNSUPPORTED"),
    (dict(max_blocks=8193), "UNSUPPORTED"), (dict(N=(1 << 20) + 1), "UNSUPPORTED"), (dict(num_pages=1 << 23), "UNSUPPORTED"),
])
def test_shapes_outside_the_contract(msa, kw, status):
    s = _shape(msa, **kw)
    for which in (msa.MSA_WS_PAGED_SPARSE_FP8, msa.MSA_WS_PAGED_DENSE_FP8):
        assert msa.msa_paged_workspace_size(s, which) == 0
    for call in CALLS:
        assert call(msa, shape=s.c())[0] == getattr(msa, "MSA_ERR_" + status)


def test_workspace_sizes(msa):
    s, p = _shape(msa), _shape(msa, prefix_blocks=3)
    sizes = [msa.msa_paged_workspace_size(s, w) for w in (msa.MSA_WS_PAGED_SPARSE_FP8, msa.MSA_WS_PAGED_DENSE_FP8)]
    assert min(sizes) > 256 and msa.msa_paged_workspace_size(p, msa.MSA_WS_PAGED_SPARSE_FP8) == sizes[0]
    assert msa.msa_paged_workspace_size(s, 6) == 0
    for call in CALLS:
        assert call(msa, ws=None)[0] == msa.MSA_ERR_WORKSPACE
        assert "aligned" in call(msa, ws=P + 128)[1]
        st, msg = call(msa, n=255)
        assert st == msa.MSA_ERR_WORKSPACE and "needed" in msg


@pytest.mark.parametrize("name", [*POOLS, "page_table", "row_start", "seq_len"])
def test_cache_pointers(msa, name):
    for bad, what in ((None, "NULL"), (P + (8 if name in POOLS else 2), "aligned")):
        c = _struct("MsaPagedCacheFp8", **{name: bad})
        for call in CALLS:
            if call is _dense and name.startswith("k_idx") or call is _read and name == "row_start":
                continue  # not used there
            st, msg = call(msa, cache=c)
            assert st == msa.MSA_ERR_INVALID_ARG and "cache." + name in msg and what in msg


def test_index_keys_are_needed_with_an_index_branch_only(msa):
    c = _struct("MsaPagedCacheFp8", k_idx=None, k_idx_exp=None)
    for call, kw in ((_sparse, dict(q_idx=None)), (_append, dict(rows=_struct("MsaNewRows", k_idx=None))), (_read, dict(k_idx=None))):
        assert "k_idx" in call(msa, cache=c)[1]
        assert call(msa, cache=c, ws=None, **kw)[0] == msa.MSA_ERR_WORKSPACE  # past the pointer checks


@pytest.mark.parametrize("call,names", [(_sparse, ("Q", "block_idx", "O", "LSE")), (_dense, ("Q", "O", "LSE")),
                                        (_read, ("out_start", "K", "V"))])
def test_pointers(msa, call, names):
    for name in names:
        st, msg = call(msa, **{name: None})
        assert st == msa.MSA_ERR_INVALID_ARG and name in msg and "NULL" in msg
        st, msg = call(msa, **{name: P + 1})
        assert st == msa.MSA_ERR_INVALID_ARG and "aligned" in msg
    for name in ("first", "k_idx"):
        if call is _read:
            assert "aligned" in call(msa, **{name: P + 1})[1]


def test_read_sizes(msa):
    assert "M=0" in _read(msa, M=0)[1] and "M=-1" in _read(msa, M=-1)[1]
    assert _read(msa, M=(1 << 28) + 1)[0] == msa.MSA_ERR_UNSUPPORTED


@pytest.mark.parametrize("bf16", [False, True])
def test_axes(msa, bf16):
    inv = msa.MSA_ERR_INVALID_ARG
    for n in (0, -1, 9, 1 << 30):
        st, msg = _append(msa, axes=_struct("MsaAxes", axes=n), bf16=bf16)
        assert st == inv and "axes" in msg
    assert "positions" in _append(msa, axes=_struct("MsaAxes", positions=None), bf16=bf16)[1]
    for name in ("positions", "axis", "axis_idx"):
        st, msg = _append(msa, axes=_struct("MsaAxes", **{name: P + 2}), bf16=bf16)
        assert st == inv and name in msg and "aligned" in msg
    # no axes at all, or all pairs on axis 0: nothing to refuse
    for axes in (None, _struct("MsaAxes", axis=None, axis_idx=None)):
        assert _append(msa, axes=axes, ws=None, bf16=bf16)[0] == msa.MSA_ERR_WORKSPACE


@pytest.mark.parametrize("bf16", [False, True])
def test_append_arguments(msa, bf16):
    for name in ("K", "V"):
        assert name in _append(msa, rows=_struct("MsaNewRows", **{name: None}), bf16=bf16)[1]
    for name in ("Q", "K", "V", "q_idx", "k_idx"):
        assert "aligned" in _append(msa, rows=_struct("MsaNewRows", **{name: P + 8}), bf16=bf16)[1]
        assert "stride of " + name in _append(msa, rows=_struct("MsaNewRows", **{"ld_" + name: 2052}), bf16=bf16)[1]
    assert "Q_out" in _append(msa, Q_out=None, bf16=bf16)[1]
    assert "rot_dim" in _append(msa, rope=_struct("MsaRope", rot_dim=24), bf16=bf16)[1]


def test_null_structs(msa):
    s, c, r, x, n = _shape(msa).c(), _struct("MsaPagedCacheFp8"), _struct("MsaRope"), _struct("MsaAxes"), _struct("MsaNewRows")
    for args in ((None, c, r, x, n), (s, None, r, x, n), (s, c, None, x, n), (s, c, r, x, None)):
        assert _call(msa, "msa_paged_append_fp8", (*args, P, P))[0] == msa.MSA_ERR_INVALID_ARG
    for name, rest in (("msa_paged_sparse_attn_fp8", 5), ("msa_paged_dense_attn_fp8", 3)):
        for args in ((None, c), (s, None)):
            assert _call(msa, name, (*args, *[P] * rest))[0] == msa.MSA_ERR_INVALID_ARG
    for args in ((None, c), (s, None)):
        assert _call(msa, "msa_paged_read_fp8", (*args, P, P, 5, P, P, P))[0] == msa.MSA_ERR_INVALID_ARG


def test_binding_refuses_caches_of_the_other_type(msa):
    one, other = msa.PagedCache.__new__(msa.PagedCache), msa.PagedCacheFp8.__new__(msa.PagedCacheFp8)
    s = _shape(msa)
    for cache, suffix in ((one, "_fp8"), (other, "")):
        calls = [(getattr(msa, "msa_paged_append" + suffix), 10), (getattr(msa, "msa_paged_sparse_attn" + suffix), 7),
                 (getattr(msa, "msa_paged_dense_attn" + suffix), 5)]
        if suffix:
            calls.append((msa.msa_paged_read_fp8, 7))
        for call, n in calls:
            with pytest.raises(TypeError, match="is needed, not a"):
                call(s, cache, *[None] * (n - 1))


def test_binding_refuses_tensors_of_another_kind(msa):
    import torch

    z = torch.zeros(2, 2, 128, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="GPU"):
        msa.PagedCacheFp8(z, z, None, None, None, None, None, None, torch.zeros(2, dtype=torch.int32))
    for n in ("K", "V", "K_exp", "V_exp", "k_idx", "k_idx_exp", "page_table", "row_start", "seq_len"):
        with pytest.raises(AttributeError, match=f"{n} of a PagedCacheFp8"):
            setattr(msa.PagedCacheFp8.__new__(msa.PagedCacheFp8), n, None)
    for n in ("axis", "axis_idx"):
        with pytest.raises(AttributeError, match=f"{n} of a Rope"):
            setattr(msa.Rope(), n, None)
    with pytest.raises(ValueError, match="GPU"):
        msa.Rope(axis=torch.zeros(4, dtype=torch.int32))


def test_reference_format_is_torchs():
    import torch

    table = torch.arange(256, dtype=torch.uint8)
    want = table.view(torch.float8_e4m3fn).double()
    got = ref8.decode(table, torch.full((), 127, dtype=torch.uint8))
    assert torch.equal(got.nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(400, 128, generator=gen) * torch.exp2(torch.randint(-110, 110, (400, 1), generator=gen).float())
    x[3], x[4, 5], x[5, 6] = 0.0, float("inf"), float("nan")
    x = x.to(torch.bfloat16)
    code, byte = ref8.quantised(x)
    scaled = torch.ldexp(x.float(), 127 - byte.int()[:, None])
    scaled = torch.where(x.isfinite(), scaled, float("nan"))
    assert torch.equal(scaled.to(torch.float8_e4m3fn).float().nan_to_num(nan=7.0), code.float().nan_to_num(nan=7.0))
    for i in range(0, 400, 7):
        want, b = ref8.encode(x[i].double().numpy())
        assert b == int(byte[i]) and (want == code[i].view(torch.uint8).numpy()).all()
        most = float(x[i].double()[x[i].isfinite()].abs().max())
        assert most <= 448 * 2.0 ** (b - 127) and (b == 10 or most > 224 * 2.0 ** (b - 127))

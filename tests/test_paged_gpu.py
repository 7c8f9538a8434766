"""The paged-cache operators on the GPU against their 64-bit forms (tests/paged_ref.py, bounds derived there)."""
import math

import numpy as np
import pytest

import paged_ref as ref

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__

    __graft_entry__.build_library()
    import block_sparse_attention_scores_gb300 as m

    return m


def _freq(rot, base=500000.0):
    import torch

    return 1.0 / base ** (torch.arange(0, rot, 2, dtype=torch.float32) / max(rot, 1))


# ----------------------------------------------------------------- append
APPEND = {
    "one": dict(counts=[1], lens=[1], Hq=8, G=2, rot=128, rot_idx=64),
    "page_ends": dict(counts=[1, 1, 1, 2, 128, 129, 3], lens=[127, 128, 129, 129, 256, 300, 3], Hq=4, G=4, rot=64, rot_idx=32),
    "idle_and_padding": dict(counts=[0, 5, 0, 0, 1, 0], lens=[7, 133, 0, 128, 500, 64], pad=3, Hq=16, G=2, rot=128, rot_idx=64),
    "interleaved": dict(counts=[3, 130], lens=[1000, 130], Hq=8, G=1, rot=128, rot_idx=64, interleaved=True),
    "partial_interleaved": dict(counts=[9], lens=[200], Hq=6, G=3, rot=48, rot_idx=16, interleaved=True),
    "partial_strided": dict(counts=[9, 4], lens=[200, 77], Hq=6, G=3, rot=96, rot_idx=48, fused=True),
    "no_rotation": dict(counts=[6], lens=[6], Hq=2, G=2, rot=0, rot_idx=0, fused=True),
    "no_index": dict(counts=[2, 2], lens=[140, 129], Hq=64, G=8, rot=128, rot_idx=0, index=False),
    "many_sequences": dict(counts=[1] * 70, lens=list(range(1, 141, 2)), Hq=2, G=1, rot=32, rot_idx=64),
    "prefill": dict(counts=[2500, 0, 37], lens=[2600, 5, 37], pad=2, Hq=2, G=1, rot=128, rot_idx=64, fused=True),
    "prefill_interleaved": dict(counts=[2433], lens=[4000], Hq=4, G=2, rot=64, rot_idx=16, interleaved=True),
    "in_place": dict(counts=[5], lens=[5], Hq=8, G=2, rot=128, rot_idx=64, in_place=True),
}


@pytest.mark.parametrize("name", APPEND)
def test_append(msa, name):
    import torch

    kw = dict(APPEND[name])
    rot, rot_idx, how = kw.pop("rot"), kw.pop("rot_idx"), kw.pop("interleaved", False)
    fused, in_place = kw.pop("fused", False), kw.pop("in_place", False)
    b = ref.Batch(stale=7.0, **kw)
    shape, cache, t = b.gpu()
    index = b.k_idx is not None
    gen = torch.Generator().manual_seed(5)
    widths = [b.Hq * 128, b.G * 128, b.G * 128] + ([b.G * 64, 64] if index else [])
    lines = torch.randn(b.N, sum(widths) + 8, generator=gen).to(torch.bfloat16).cuda()[:, :sum(widths)]
    parts = list(lines.split(widths, dim=1)) if fused else [x.contiguous() for x in lines.split(widths, dim=1)]
    x = dict(zip(("Q", "K", "V", "q_idx", "k_idx"),
                 [p.unflatten(1, s) for p, s in zip(parts, [(b.Hq, 128), (b.G, 128), (b.G, 128), (b.G, 64), (64,)])]))
    was = {n: v.clone() for n, v in x.items()}
    f, fi = _freq(rot), _freq(rot_idx)
    rope = msa.Rope(f.cuda(), fi.cuda() if index else None, interleaved=how)
    out = x["Q"] if in_place else torch.full((b.N, b.Hq, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    qi_out = None
    if index:
        qi_out = x["q_idx"] if in_place else torch.full((b.N, b.G, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_APPEND)
    msa.msa_paged_append(shape, cache, rope, x["K"], x["V"], x.get("k_idx"), x["Q"], x.get("q_idx"), out, qi_out, ws)
    msa.msa_check_device_status(ws)

    # a result is a rounding of sums of two products with fp32 sin and cos: 2^-8 of it and 2^-20 of |a| + |b|
    def close(got, y, mag, what):
        assert bool(((got.double() - y).abs() <= 2.0 ** -8 * y.abs() + 2.0 ** -20 * mag).all()), what

    want = {n: getattr(b, n).clone() for n in ("K", "V", "k_idx") if getattr(b, n) is not None}
    got = {n: t[n].cpu() for n in want}
    src = {n: v.cpu() for n, v in was.items()}
    for r in range(b.n):
        page, slot = int(b.table[b.row_seq[r], b.row_pos[r] // 128]), b.row_pos[r] % 128
        for n in ("K", "V", "k_idx"):
            if n not in want:
                continue
            here = (page, slice(None), slot) if n != "k_idx" else (page, slot)
            y, mag = ref.rotated(src[n][r].double(), b.row_pos[r], fi if n == "k_idx" else f, how)
            if n == "V":
                y, mag = src[n][r].double(), 0.0 * mag
            close(got[n][here], y, mag, (n, r))
            got[n][here] = want[n][here]
        close(out[r].cpu(), *ref.rotated(src["Q"][r].double(), b.row_pos[r], f, how), ("Q", r))
        if index:
            close(qi_out[r].cpu(), *ref.rotated(src["q_idx"][r].double(), b.row_pos[r], fi, how), ("q_idx", r))
    for n in want:  # nothing else of the pools was touched
        assert torch.equal(got[n], want[n]), n
    rest = src["Q"][b.n:] if in_place else torch.full_like(src["Q"][b.n:], 3.0)
    assert torch.equal(out[b.n:].cpu(), rest)


def test_append_far_positions(msa):
    """Angles at positions up to 2^20 - 1, where a product in fp32 would be off by 0.06 radians."""
    import torch

    pos = [0, 1, 4095, 99999, 524287, 1048574, 1048575]
    S, G, Hq = len(pos), 1, 1
    table = torch.arange(S, dtype=torch.int32).repeat_interleave(8192).view(S, 8192).cuda()
    K, V = (torch.zeros(S, G, 128, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache = msa.PagedCache(K, V, None, table, torch.arange(S + 1, dtype=torch.int32, device="cuda"),
                           torch.tensor([p + 1 for p in pos], dtype=torch.int32, device="cuda"))
    shape = msa.PagedShape(S=S, N=S, Hq=Hq, G=G, num_pages=S, max_blocks=8192)
    new = torch.randn(S, 1, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    for f in (_freq(128), torch.linspace(-3.0, 40.0, 64)):  # frequencies past one turn, and backward ones, too
        ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_APPEND)
        Q, _ = msa.paged_append(shape, cache, msa.Rope(f.cuda()), new, new, Q=new, workspace=ws)
        msa.msa_check_device_status(ws)
        for r, p in enumerate(pos):
            y, mag = ref.rotated(new[r].cpu().double(), p, f, False)
            # the phase is kept to 2^-32 turns and rounded to fp32 (pi 2^-24), sin and cos to fp32
            bound = 2.0 ** -8 * y.abs() + 2.0 ** -20 * mag
            assert bool(((Q[r].cpu().double() - y).abs() <= bound).all()), p
            assert bool(((K[r, :, p % 128].cpu().double() - y).abs() <= bound).all()), p


# ----------------------------------------------------------------- sparse
SPARSE = {
    "first_token": dict(counts=[1], lens=[1], Hq=8, G=2, k=4),
    "page_ends": dict(counts=[1, 1, 1, 1, 1, 1], lens=[2, 127, 128, 129, 256, 257], Hq=8, G=2, k=2),
    "k1": dict(counts=[1, 2], lens=[700, 1300], Hq=4, G=2, k=1),
    "hg1_g3": dict(counts=[2, 1], lens=[1500, 2000], Hq=3, G=3, k=5),
    "hg2_idle_padding": dict(counts=[0, 3, 0, 1], lens=[50, 1027, 0, 4000], Hq=4, G=2, k=7, pad=2),
    "hg8_rows": dict(counts=[5, 1, 9], lens=[5000, 640, 900], Hq=16, G=2, k=16),
    "g8": dict(counts=[1, 1, 2], lens=[3000, 2999, 5111], Hq=32, G=8, k=16),
    "all_blocks_kept": dict(counts=[1, 4], lens=[1000, 260], Hq=8, G=1, k=40),
    "k33": dict(counts=[1, 1], lens=[9000, 8193], Hq=4, G=1, k=33),
    "k128": dict(counts=[2], lens=[128 * 140 + 5], Hq=2, G=1, k=128),
    "many_rows": dict(counts=[40, 1, 30], lens=[2040, 1, 1037], Hq=8, G=2, k=4),
}


def _sparse(msa, b, k, **kw):
    import torch

    shape, cache, t = b.gpu(k)
    ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_SPARSE)
    ws.fill_(255)  # no result may depend on what a workspace held
    bi = torch.full((b.N, b.G, k), -7, dtype=torch.int32, device="cuda")
    O = torch.full((b.N, b.Hq, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    LSE = torch.full((b.N, b.Hq), 5.0, device="cuda")
    msa.msa_paged_sparse_attn(shape, cache, t["Q"], t["q_idx"], bi, O, LSE, ws, **kw)
    msa.msa_check_device_status(ws)
    return O.cpu(), LSE.cpu(), bi.cpu().numpy()


def _check_padding(b, O, LSE, bi=None):
    assert bool((O[b.n:] == 5.0).all()) and bool((LSE[b.n:] == 5.0).all())
    assert bi is None or (bi[b.n:] == -7).all()


@pytest.mark.parametrize("stale", [NAN, INF, 3e38], ids=["nan", "inf", "huge"])
@pytest.mark.parametrize("name", SPARSE)
def test_sparse(msa, name, stale):
    kw = dict(SPARSE[name])
    k = kw.pop("k")
    b = ref.Batch(stale=stale, seed=3, **kw)
    O, LSE, bi = _sparse(msa, b, k)
    for r in range(b.n):
        np.testing.assert_array_equal(bi[r], ref.select(b, r, k), err_msg=f"row {r}")
    rows = range(b.n) if b.n < 20 else range(0, b.n, 5)
    ref.check_attention(b, rows, range(b.Hq), O, LSE, lambda r, g: bi[r, g].tolist())
    _check_padding(b, O, LSE, bi)


def test_sparse_long(msa):
    """A quarter of a million tokens, two rows: more blocks than a pass of the selection's threads."""
    b = ref.Batch(counts=[2], lens=[1 << 18], Hq=2, G=1, seed=8)
    O, LSE, bi = _sparse(msa, b, 16)
    for r in range(2):
        np.testing.assert_array_equal(bi[r], ref.select(b, r, 16))
    ref.check_attention(b, range(2), range(2), O, LSE, lambda r, g: bi[r, g].tolist())


@pytest.mark.parametrize("k", [2, 4, 9])
def test_selection_at_narrow_borders(msa, k):
    """Blocks that fp32 sums cannot tell apart: exact ties (equal pages, equal rows in another order) go to the lower
    id, and gaps of 2^-26 of the score are decided as they are."""
    import torch

    b = ref.Batch(counts=[1, 3], lens=[128 * 24 + 40, 128 * 24 + 3], Hq=2, G=2, seed=11)
    gen = torch.Generator().manual_seed(2)
    for s in range(2):
        first = b.k_idx[b.table[s, 0].long()].clone()
        for c in range(1, 24):
            page = int(b.table[s, c])
            if c % 3 == 0:
                b.k_idx[page] = first                                   # the same page again
            elif c % 3 == 1:
                b.k_idx[page] = first[torch.randperm(128, generator=gen)]  # its keys in another order
            else:
                b.k_idx[page] = first
                # every key's dim e moves by a value far below the score's fp32 step
                e = int(torch.randint(0, 64, (1,), generator=gen))
                b.k_idx[page, :, e] = first[:, e] * (1 + 2.0 ** -7 * int(torch.randint(-1, 2, (1,), generator=gen)))
                b.q_idx[:, :, e] = (b.q_idx[:, :, e].float() * 2.0 ** -18).to(torch.bfloat16)
    _, _, bi = _sparse(msa, b, k)
    for r in range(b.n):
        np.testing.assert_array_equal(bi[r], ref.select(b, r, k), err_msg=f"row {r}")


def test_selection_with_one_large_component(msa):
    """One product of a score dwarfs the others, which a sum that starts with it cuts off: what decides between the
    blocks lies below its fp32 step."""
    import torch

    b = ref.Batch(counts=[2, 1], lens=[128 * 60 + 9, 128 * 77], Hq=2, G=2, seed=14)
    gen = torch.Generator().manual_seed(3)

    def small(*shape):
        return (2.0 ** -12 * (1 + torch.rand(*shape, generator=gen))).to(torch.bfloat16)

    for s in range(2):
        for c in range(60 + 17 * s):
            b.k_idx[int(b.table[s, c])] = small(128, 64)
            b.k_idx[int(b.table[s, c]), :, 0] = 1.0
    b.q_idx[:b.n] = small(b.n, 2, 64)
    b.q_idx[:b.n, :, 0] = 1.0
    _, _, bi = _sparse(msa, b, 9)
    for r in range(b.n):
        np.testing.assert_array_equal(bi[r], ref.select(b, r, 9), err_msg=f"row {r}")


def test_selection_with_nan_and_infinite_index_values(msa):
    """A NaN score counts as -infinity; infinite scores order as they are; huge ones do not overflow."""
    b = ref.Batch(counts=[1, 2, 1, 1], lens=[128 * 12 + 7] * 4, Hq=2, G=2, seed=12)
    for s, v in ((0, NAN), (1, INF), (2, 2e38)):
        b.k_idx[int(b.table[s, 3]), 5] = v
        b.k_idx[int(b.table[s, 7]), :, 9] = v
        b.k_idx[int(b.table[s, 8]), 100] = -v
    b.q_idx[4, 0, 3] = NAN  # every score of this (row, group)
    b.q_idx[4, 1] = 0.0     # every score zero: the lowest ids
    _, _, bi = _sparse(msa, b, 4)
    for r in range(b.n):
        np.testing.assert_array_equal(bi[r], ref.select(b, r, 4), err_msg=f"row {r}")


def test_sparse_with_a_given_selection(msa):
    """IndexShare: block_idx is read; no index keys are needed; an empty list gives O = 0 and LSE = -infinity."""
    import torch

    b = ref.Batch(counts=[1, 3, 0, 2], lens=[1000, 2000, 9, 130], Hq=8, G=2, seed=4, index=False, pad=1)
    k = 6
    rng = np.random.default_rng(0)
    bi = np.full((b.N, b.G, k), -1, np.int32)
    for r in range(b.n):
        for g in range(b.G):
            last = b.row_pos[r] // 128
            ids = sorted(rng.choice(last, min(last, k - 1), replace=False).tolist() + [last]) if last else [0]
            bi[r, g, :len(ids)] = ids
    bi[1, 0] = -1                     # nothing selected
    bi[2, 1] = [0, 3, -1, -1, -1, -1]  # without the own block
    shape, cache, t = b.gpu(k)
    ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_SPARSE)
    O, LSE, _ = msa.paged_sparse_attn(shape, cache, t["Q"], block_idx=torch.from_numpy(bi).cuda(), workspace=ws)
    msa.msa_check_device_status(ws)
    ref.check_attention(b, range(b.n), range(b.Hq), O.cpu(), LSE.cpu(), lambda r, g: bi[r, g].tolist())
    assert float(LSE[1, 0]) == -INF and bool((O[1, :4] == 0).all())


# ----------------------------------------------------------------- dense
DENSE = {
    "first_token": dict(counts=[1], lens=[1], Hq=8, G=2),
    "page_ends": dict(counts=[1, 1, 1, 1, 1], lens=[127, 128, 129, 256, 257], Hq=8, G=2),
    "rows_hg1": dict(counts=[20, 3, 17], lens=[20, 131, 400], Hq=3, G=3),
    "rows_hg2_idle": dict(counts=[0, 7, 0, 1], lens=[0, 300, 77, 900], Hq=4, G=2, pad=2),
    "rows_hg4": dict(counts=[9, 1, 5], lens=[1000, 2, 133], Hq=8, G=2),
    "rows_hg8": dict(counts=[3, 4], lens=[1500, 260], Hq=16, G=2),
    "g8_long": dict(counts=[1, 2], lens=[7000, 6001], Hq=32, G=8),
    "prefix1": dict(counts=[1, 1], lens=[129, 200], Hq=8, G=2, prefix=1),
    "prefix_hg1": dict(counts=[1, 3, 0, 2], lens=[128 * 5 + 1, 128 * 5 + 300, 9, 128 * 5 + 2], Hq=3, G=3, prefix=5, pad=1),
    "prefix_hg2": dict(counts=[2, 1], lens=[128 * 9 + 2, 128 * 9 + 128], Hq=2, G=1, prefix=9),
    "prefix_hg4_rows": dict(counts=[1] * 30 + [4] * 11, lens=[128 * 12 + 4 + i for i in range(41)], Hq=8, G=2, prefix=12),
    "prefix_hg8": dict(counts=[1] * 21, lens=[128 * 40 + 1 + 9 * i for i in range(21)], Hq=16, G=2, prefix=40),
    "prefix_two_pairs": dict(counts=[5] * 20, lens=[128 * 6 + 7 + 3 * i for i in range(20)], Hq=32, G=8, prefix=6),
    "prefix_idle_first": dict(counts=[0, 1, 2], lens=[0, 128 * 3 + 5, 128 * 3 + 9], Hq=4, G=1, prefix=3),
}


def _dense(msa, b, **kw):
    import torch

    shape, cache, t = b.gpu()
    ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_DENSE)
    ws.fill_(255)
    O = torch.full((b.N, b.Hq, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    LSE = torch.full((b.N, b.Hq), 5.0, device="cuda")
    msa.msa_paged_dense_attn(shape, cache, t["Q"], O, LSE, ws, **kw)
    msa.msa_check_device_status(ws)
    return O.cpu(), LSE.cpu()


def _all(b):
    return lambda r, g: list(range(b.row_pos[r] // 128 + 1))


@pytest.mark.parametrize("stale", [NAN, INF], ids=["nan", "inf"])
@pytest.mark.parametrize("name", DENSE)
def test_dense(msa, name, stale):
    b = ref.Batch(stale=stale, seed=6, **DENSE[name])
    O, LSE = _dense(msa, b)
    rows = range(b.n) if b.n < 30 else range(0, b.n, 7)
    heads = range(b.Hq) if b.Hq <= 8 else range(0, b.Hq, 5)
    ref.check_attention(b, rows, heads, O, LSE, _all(b), bf16_p=b.prefix > 0)
    _check_padding(b, O, LSE)


# Shared prefixes of enough pages (counted for every sequence and group) to be read once for the batch.
PREFIX = {
    "hg1": dict(counts=[1, 3, 0, 2] * 5, lens=[128 * 40 + 3 + 9 * i for i in range(20)], Hq=2, G=2, prefix=40, pad=1),
    "hg2": dict(counts=[2, 1, 1] * 10, lens=[128 * 26 + 2 + 41 * i for i in range(30)], Hq=4, G=2, prefix=26),
    "hg4": dict(counts=[0] + [1, 2] * 12 + [1], lens=[7] + [128 * 60 + 2 + 17 * i for i in range(25)], Hq=4, G=1, prefix=60),
    "hg8": dict(counts=[1] * 16, lens=[128 * 100 + 1 + 64 * i for i in range(16)], Hq=8, G=1, prefix=100, pad=2),
    "three_pairs": dict(counts=[1] * 70, lens=[128 * 12 + 1 + i for i in range(70)], Hq=16, G=2, prefix=12),
}


@pytest.mark.parametrize("stale", [NAN, INF], ids=["nan", "inf"])
@pytest.mark.parametrize("name", PREFIX)
def test_dense_prefix(msa, name, stale):
    b = ref.Batch(stale=stale, seed=26, **PREFIX[name])
    assert b.S * b.prefix * b.G > 1500 and b.N * b.hg <= 9 * b.S
    O, LSE = _dense(msa, b)
    rows = range(0, b.n, 1 if b.n < 30 else 7)
    ref.check_attention(b, rows, range(b.Hq) if b.Hq <= 8 else range(0, b.Hq, 5), O, LSE, _all(b), bf16_p=True)
    _check_padding(b, O, LSE)


def test_dense_prefix_large_scores(msa):
    b = ref.Batch(counts=[2, 1] * 20, lens=[128 * 20 + 90 + 3 * i for i in range(40)], Hq=8, G=2, prefix=20, seed=9)
    for c in range(20):
        b.K[int(b.table[0, c])] *= float(1 + 3 * (c % 7))
    b.Q *= 4
    O, LSE = _dense(msa, b)
    ref.check_attention(b, range(0, b.n, 5), range(b.Hq), O, LSE, _all(b), bf16_p=True)


def test_dense_prefix_bad_batches(msa):
    def run(change, good):
        b = ref.Batch(counts=[1] * 20, lens=[128 * 40 + 3 + 9 * i for i in range(20)], Hq=8, G=2, prefix=40, seed=1)
        change(b)
        shape, cache, t = b.gpu()
        ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_DENSE)
        ws.fill_(255)
        O, LSE = msa.paged_dense_attn(shape, cache, t["Q"], workspace=ws)
        with pytest.raises(msa.MsaError) as e:
            msa.msa_check_device_status(ws)
        assert e.value.status == msa.MSA_ERR_DEVICE
        ref.check_attention(b, good, range(0, 8, 3), O.cpu(), LSE.cpu(), _all(b), bf16_p=True)

    def everywhere(c, v):
        return lambda b: b.table.__setitem__((slice(None), c), v)

    for v in (-1, 1 << 20, 2 ** 31 - 1, -2 ** 31):
        run(everywhere(17, v), [])                                         # a bad page of the prefix
        run(lambda b: b.table.__setitem__((3, 40), v), [0, 2, 4, 19])      # of a sequence's own
        run(lambda b: b.lens.__setitem__(5, v if v < 0 else 128 * 40), [0, 4, 6, 19])  # no row, or one inside the prefix
    run(lambda b: b.table.__setitem__((7, 11), b.table[7, 12]), [])       # a prefix that is not shared


def test_dense_prefix_same_bits(msa):
    """Again, beside itself on another stream, and from a graph."""
    import torch

    b = ref.Batch(counts=[1] * 14, lens=[128 * 30 + 5 + 37 * i for i in range(14)], Hq=16, G=4, prefix=30, seed=2)
    want = _dense(msa, b)
    shape, cache, t = b.gpu()
    ws = [msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_DENSE) for _ in range(2)]
    out = [(torch.zeros_like(t["Q"]), torch.zeros(b.N, b.Hq, device="cuda")) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for w, (O, LSE), s in zip(ws, out, streams):
            msa.msa_paged_dense_attn(shape, cache, t["Q"], O, LSE, w, s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in (0, 1, 0):
            msa.msa_paged_dense_attn(shape, cache, t["Q"], *out[i], ws[0])
    for again in range(3):
        for w, (O, LSE) in zip(ws, out):
            msa.msa_check_device_status(w)
            assert torch.equal(O.cpu(), want[0]) and torch.equal(LSE.cpu(), want[1]), again
            O.zero_()
            LSE.zero_()
        g.replay()
        torch.cuda.synchronize()


@pytest.mark.parametrize("stale", [NAN, INF], ids=["nan", "inf"])
@pytest.mark.parametrize("counts,lens,Hq,G,prefix", [([127], [128 * 60 + 127], 16, 2, 60), ([16], [128 * 200 + 50], 8, 1, 200),
                                                     ([40, 0, 9], [128 * 30 + 128, 4, 128 * 30 + 77], 24, 3, 30)], ids=str)
def test_dense_chunk_of_a_page_behind_a_prefix(msa, counts, lens, Hq, G, prefix, stale):
    """Many rows of a sequence whose own part is one page: the pages before it are read once for all of them."""
    b = ref.Batch(counts=counts, lens=lens, Hq=Hq, G=G, prefix=prefix, seed=27, stale=stale, pad=1)
    before = msa.msa_kernel_launches()
    O, LSE = _dense(msa, b)
    assert msa.msa_kernel_launches() - before == 4  # rows, prefix, own pages, merge
    ref.check_attention(b, range(0, b.n, 5), range(0, b.Hq, 3), O, LSE, _all(b), bf16_p=True)
    _check_padding(b, O, LSE)


# Several rows per sequence: more than eight columns on average and more than a page take 128-row tiles (of 128 / h_g
# rows, two at a time).
RUNS = {
    "hg8": dict(counts=[5, 3, 8], lens=[700, 130, 1000], Hq=16, G=2),
    "one_group": dict(counts=[4, 9], lens=[513, 900], Hq=8, G=1),
    "two_tiles": dict(counts=[20, 33, 1], lens=[600, 400, 300], Hq=16, G=2, pad=3),
    "two_tiles_one_group": dict(counts=[17, 40], lens=[17, 390], Hq=8, G=1),
    "hg1": dict(counts=[300, 10, 0, 129], lens=[1000, 300, 50, 129], Hq=2, G=2),
    "hg2_three_groups": dict(counts=[6, 70], lens=[256, 500], Hq=6, G=3),
    "hg4_ends": dict(counts=[4, 4, 4, 4, 4], lens=[127, 128, 130, 256, 259], Hq=8, G=2),
    "long": dict(counts=[4], lens=[128 * 70 + 2], Hq=16, G=2),
    "long_across_pages": dict(counts=[16], lens=[128 * 30 + 7], Hq=8, G=1),
    "prefix": dict(counts=[3, 18, 0, 5], lens=[128 * 6 + 3, 128 * 6 + 400, 4, 128 * 7 + 5], Hq=16, G=2, prefix=6),
    "prefix_three_pairs": dict(counts=[7] * 13, lens=[128 * 3 + 7 + 11 * i for i in range(13)], Hq=24, G=3, prefix=3),
    "prefix_hg1_one_group": dict(counts=[12, 140], lens=[128 * 2 + 12, 128 * 2 + 300], Hq=1, G=1, prefix=2, pad=2),
}


@pytest.mark.parametrize("stale", [NAN, INF], ids=["nan", "inf"])
@pytest.mark.parametrize("name", RUNS)
def test_dense_rows(msa, name, stale):
    b = ref.Batch(stale=stale, seed=16, **RUNS[name])
    O, LSE = _dense(msa, b)
    rows = range(b.n) if b.n < 60 else range(0, b.n, 7)
    heads = range(b.Hq) if b.Hq <= 8 else range(0, b.Hq, 5)
    ref.check_attention(b, rows, heads, O, LSE, _all(b), bf16_p=b.prefix > 0)
    _check_padding(b, O, LSE)


@pytest.mark.parametrize("shape", [dict(counts=[6, 5], lens=[262, 140], Hq=16, G=2),
                                   dict(counts=[20, 9], lens=[400, 134], Hq=8, G=1),
                                   dict(counts=[140, 9], lens=[400, 262], Hq=3, G=3),
                                   dict(counts=[6, 5], lens=[520, 515], Hq=16, G=2, prefix=3)], ids=str)
def test_later_rows_do_not_reach_earlier_ones_of_a_tile(msa, shape):
    """As above for 128-row tiles; and the rows that see such values have them: those of V as they are added up."""
    import torch

    b = ref.Batch(seed=10, **shape)
    clean = _dense(msa, b)
    # the sequence's last but i row: NaN, infinities of one and of both signs in V alone; NaN in K and V
    for s in range(2):
        for i, d, v in ((0, 3, NAN), (1, 40, INF), (2, 70, -INF), (2, 90, INF), (3, 90, -INF)):
            t = b.lens[s] - 1 - i
            b.V[int(b.table[s, t // 128]), :, t % 128, d] = v
    O, LSE = _dense(msa, b)
    assert bool((LSE[:b.n] == clean[1][:b.n]).all())
    for r in range(b.n):
        want = clean[0][r].clone()
        behind = b.lens[b.row_seq[r]] - 1 - b.row_pos[r]
        if behind <= 3:
            want[:, 90] = -INF
        if behind <= 2:
            want[:, 70], want[:, 90] = -INF, NAN
        if behind <= 1:
            want[:, 40] = INF
        if behind <= 0:
            want[:, 3] = NAN
        same = (O[r] == want) | (O[r].isnan() & want.isnan())
        assert bool(same.all()), (r, behind, torch.nonzero(~same)[:4].tolist())
    for s in range(2):
        t = b.lens[s] - 1 - 2
        b.K[int(b.table[s, t // 128]), :, t % 128] = NAN
    O, LSE = _dense(msa, b)
    for r in range(b.n):
        behind = b.lens[b.row_seq[r]] - 1 - b.row_pos[r]
        if behind > 3:
            assert bool((O[r] == clean[0][r]).all()) and bool((LSE[r] == clean[1][r]).all()), r
        elif behind <= 2:
            assert bool(O[r].isnan().all()) and bool(LSE[r].isnan().all()), r


def test_dense_rows_large_scores(msa):
    b = ref.Batch(counts=[3, 2, 20], lens=[128 * 6 + 90, 128 * 7, 128 * 6 + 1], Hq=16, G=2, seed=9)
    for s in range(3):
        for c in range(6):
            b.K[int(b.table[s, c])] *= 1.0 if s else float(1 + 3 * c)
    b.Q *= 4
    O, LSE = _dense(msa, b)
    ref.check_attention(b, range(b.n), range(0, b.Hq, 3), O, LSE, _all(b))


def _shared_pages(S, rows, length, Hq, G, seed=21):
    """A batch whose sequences all have the same pages (nothing is appended here, so they may)."""
    one = ref.Batch(counts=[rows], lens=[length], Hq=Hq, G=G, seed=seed)
    b = ref.Batch(counts=[rows] * S, lens=[0] * S, Hq=Hq, G=G, seed=seed + 1, spare=0, index=False)
    b.K, b.V, b.k_idx, b.num_pages, b.max_blocks = one.K, one.V, one.k_idx, one.num_pages, one.max_blocks
    b.table, b.lens = one.table.expand(S, -1).contiguous(), [length] * S
    b.row_pos = [length - rows + j for _ in range(S) for j in range(rows)]
    return b


def test_dense_rows_many_long(msa):
    """So many sequences that a run has all their pages: more than the 32 that are looked up at a time."""
    b = _shared_pages(1530, 2, 128 * 69 + 5, 8, 1)
    O, LSE = _dense(msa, b)
    ref.check_attention(b, [0, 1, 700, 1531, 3059], range(0, 8, 3), O, LSE, _all(b))


def test_dense_single_rows_many_long(msa):
    b = _shared_pages(1600, 1, 128 * 69 + 5, 8, 1)
    O, LSE = _dense(msa, b)
    ref.check_attention(b, [0, 1, 700, 1599], range(0, 8, 3), O, LSE, _all(b))


@pytest.mark.parametrize("S,rows,Hq,G", [(4500, 1, 2, 1), (2100, 3, 2, 1), (700, 3, 8, 1), (1, 1200, 2, 2)], ids=str)
def test_many_sequences_and_rows(msa, S, rows, Hq, G):
    """More sequences than are kept in shared memory, and more rows than a pass over them takes."""
    b = _shared_pages(S, rows, max(rows, 200), Hq, G)
    O, LSE = _dense(msa, b)
    some = sorted({0, 1, 300, 1023, 1024, 1025, 1100, b.n - 2, b.n - 1})
    ref.check_attention(b, some, range(Hq), O, LSE, _all(b))
    O, LSE, bi = _sparse(msa, b, 2)
    for r in some:
        np.testing.assert_array_equal(bi[r], ref.select(b, r, 2))
    ref.check_attention(b, some, range(Hq), O, LSE, lambda r, g: bi[r, g].tolist())


def test_sparse_whole_rows_many(msa):
    """More selected blocks in a row's run than the 32 that are looked up at a time."""
    b = _shared_pages(1600, 1, 128 * 69 + 5, 2, 1)
    O, LSE, bi = _sparse(msa, b, 100)
    for r in (0, 5, 1599):
        np.testing.assert_array_equal(bi[r], ref.select(b, r, 100))
    ref.check_attention(b, [0, 5, 1599], range(2), O, LSE, lambda r, g: bi[r, g].tolist())


@pytest.mark.parametrize("k,lens", [(1, [700] * 90), (3, [128] * 200), (4, [128 * 9 + 3] * 90), (1, [5])], ids=str)
def test_workspaces_of_the_least_size(msa, k, lens):
    """Calls that need no block maxima, or no parts, leave what lies behind their workspace alone."""
    import torch

    b = ref.Batch(counts=[1] * len(lens), lens=lens, Hq=8, G=2, seed=36)
    shape, cache, t = b.gpu(k)
    for which in (msa.MSA_WS_PAGED_SPARSE, msa.MSA_WS_PAGED_DENSE):
        n = msa.msa_paged_workspace_size(shape, which)
        buf = torch.full((n + (1 << 20),), 255, dtype=torch.uint8, device="cuda")
        if which == msa.MSA_WS_PAGED_SPARSE:
            O, LSE, bi = msa.paged_sparse_attn(shape, cache, t["Q"], t["q_idx"], workspace=buf[:n])
            for r in (0, b.n - 1):
                np.testing.assert_array_equal(bi[r].cpu().numpy(), ref.select(b, r, k))
            blocks = (lambda r, g: bi[r, g].tolist())
        else:
            O, LSE = msa.paged_dense_attn(shape, cache, t["Q"], workspace=buf[:n])
            blocks = _all(b)
        msa.msa_check_device_status(buf)
        ref.check_attention(b, sorted({0, b.n // 2, b.n - 1}), range(8), O.cpu(), LSE.cpu(), blocks)
        assert bool((buf[n:] == 255).all())


def test_sparse_prompt(msa):
    """A prompt's thousands of rows (and a single one beside it): a page's scores take as many columns as rows and groups."""
    b = ref.Batch(counts=[4000, 1], lens=[128 * 40 + 3, 128 * 33], Hq=8, G=4, seed=35, pad=2)
    O, LSE, bi = _sparse(msa, b, 4)
    some = [0, 1, 127, 128, 1999, 3990, 3999, 4000]
    for r in some:
        np.testing.assert_array_equal(bi[r], ref.select(b, r, 4), err_msg=f"row {r}")
    ref.check_attention(b, some, range(8), O, LSE, lambda r, g: bi[r, g].tolist())
    _check_padding(b, O, LSE, bi)


@pytest.mark.parametrize("blocks", [256, 257, 258, 2049, 2050])
def test_selection_threads_change(msa, blocks):
    """Page tables of the widths around which the selection's block of threads grows."""
    b = ref.Batch(counts=[1, 1], lens=[128 * blocks, 128 * (blocks - 1) + 1], Hq=1, G=1, seed=19)
    assert b.max_blocks == blocks
    O, LSE, bi = _sparse(msa, b, 7)
    for r in range(2):
        np.testing.assert_array_equal(bi[r], ref.select(b, r, 7))
    ref.check_attention(b, range(2), range(1), O, LSE, lambda r, g: bi[r, g].tolist())


@pytest.mark.parametrize("Hq,pad,prefix", [(16, 4, 0), (16, 4, 2), (2, 1, 2), (2, 1, 0)], ids=str)
def test_batch_without_rows(msa, Hq, pad, prefix):
    """Idle slots and padded rows only: outputs and pools as they were."""
    import torch

    b = ref.Batch(counts=[0, 0, 0], lens=[0, 300, 128 * 5], Hq=Hq, G=2, pad=pad, prefix=prefix, seed=3)
    O, LSE = _dense(msa, b)
    assert bool((O == 5).all()) and bool((LSE == 5).all())
    O, LSE, bi = _sparse(msa, b, 3)
    assert bool((O == 5).all()) and bool((LSE == 5).all()) and bool((bi == -7).all())
    shape, cache, t = b.gpu()
    before = t["K"].clone().view(torch.int16)
    ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_APPEND)
    new = torch.ones(b.N, 2, 128, dtype=torch.bfloat16, device="cuda")
    msa.paged_append(shape, cache, msa.Rope(), new, new, workspace=ws)
    msa.msa_check_device_status(ws)
    assert torch.equal(t["K"].view(torch.int16), before)


@pytest.mark.parametrize("S,rows", [(5000, 1), (2500, 2)], ids=str)
def test_prefix_of_more_rows_than_a_wave(msa, S, rows):
    """More pairs of row tiles than SMs."""
    b = _shared_pages(S, rows, 128 * 4 + 9, 8, 1)
    b.prefix = 2
    O, LSE = _dense(msa, b)
    some = [0, 1, 31, 32, 2047, 4865, b.n - 1]
    ref.check_attention(b, some, range(0, 8, 3), O, LSE, _all(b), bf16_p=True)


def test_dense_rows_bad_batches(msa):
    """Several rows per sequence: faults of one sequence are reported and leave the others alone."""
    import torch

    def run(change, good, prefix=0):
        b = ref.Batch(counts=[3, 4, 20], lens=[128 * 5 + 2, 128 * 6 + 9, 128 * 4 + 60], Hq=16, G=2, prefix=prefix, seed=1)
        change(b)
        shape, cache, t = b.gpu()
        ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_DENSE)
        ws.fill_(255)
        O, LSE = msa.paged_dense_attn(shape, cache, t["Q"], workspace=ws)
        with pytest.raises(msa.MsaError) as e:
            msa.msa_check_device_status(ws)
        assert e.value.status == msa.MSA_ERR_DEVICE
        ref.check_attention(b, good, range(0, 16, 5), O.cpu(), LSE.cpu(), _all(b), bf16_p=prefix > 0)

    def page(s, c, v):
        return lambda b: b.table.__setitem__((s, c), v)

    def length(s, v):
        return lambda b: b.lens.__setitem__(s, v)

    for v in (-1, 1 << 20, 2 ** 31 - 1, -2 ** 31):
        run(page(0, 5, v), [3, 6, 7, 26])
        run(page(0, 2, v), [3, 6, 7, 26])
        run(page(2, 4, v), [0, 2, 3, 6], prefix=2)
    for v in (0, -5, 2, 128 * 7 + 1, 2 ** 31 - 1, -2 ** 31):
        run(length(1, v), [0, 2, 7, 26])
        run(length(1, v), [0, 2, 7, 26], prefix=2)
    run(lambda b: b.table.__setitem__((1, 1), b.table[1, 3]), [], prefix=2)  # a prefix that is not shared


def test_dense_rows_same_bits(msa):
    """Again, on another stream beside another call, and from a graph that is replayed on another batch."""
    import torch

    args = dict(counts=[5, 0, 33, 2, 9], Hq=16, G=2, prefix=2, pad=2)
    b = ref.Batch(lens=[128 * 5 + 9, 0, 128 * 3 + 40, 128 * 9, 128 * 12 + 77], seed=4, **args)
    want = _dense(msa, b)
    shape, cache, t = b.gpu()
    ws = [msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_DENSE) for _ in range(2)]
    out = [(torch.full_like(t["Q"], 5.0), torch.full((b.N, b.Hq), 5.0, device="cuda")) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for w, (O, LSE), s in zip(ws, out, streams):
            msa.msa_paged_dense_attn(shape, cache, t["Q"], O, LSE, w, s)
    torch.cuda.synchronize()
    for w, (O, LSE) in zip(ws, out):
        msa.msa_check_device_status(w)
        assert torch.equal(O[:b.n].cpu(), want[0][:b.n]) and torch.equal(LSE[:b.n].cpu(), want[1][:b.n])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        msa.msa_paged_dense_attn(shape, cache, t["Q"], *out[0], ws[0])
        msa.msa_paged_dense_attn(shape, cache, t["Q"], *out[1], ws[0])
    # other rows of the same shape: fewer, elsewhere
    counts, lens = [1, 20, 0, 18, 10], [128 * 4, 128 * 3 + 20, 7, 128 * 8 + 99, 128 * 12 + 1]
    starts = np.cumsum([0] + counts)
    cache.row_start.copy_(torch.tensor(starts, dtype=torch.int32))
    cache.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
    table = b.table.clone()
    table[1, :4] = torch.tensor([int(table[0, 0]), int(table[0, 1]), int(table[4, 5]), int(table[4, 6])])
    cache.page_table.copy_(table)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    msa.msa_check_device_status(ws[0])
    b.table, b.lens, b.counts, b.n = table, lens, counts, int(starts[-1])
    b.row_seq = [i for i, c in enumerate(counts) for _ in range(c)]
    b.row_pos = [x - c + j for c, x in zip(counts, lens) for j in range(c)]
    for O, LSE in out:
        ref.check_attention(b, range(0, b.n, 2), range(0, 16, 5), O.cpu(), LSE.cpu(), _all(b), bf16_p=True)
    assert torch.equal(out[0][0][:b.n], out[1][0][:b.n])


def test_sparse_half_a_million(msa):
    """More blocks than the selection's smaller block of threads holds."""
    b = ref.Batch(counts=[1], lens=[(1 << 19) - 3], Hq=2, G=1, seed=18)
    O, LSE, bi = _sparse(msa, b, 16)
    np.testing.assert_array_equal(bi[0], ref.select(b, 0, 16))
    ref.check_attention(b, [0], range(2), O, LSE, lambda r, g: bi[r, g].tolist())


@pytest.mark.parametrize("what", ["zero queries", "zero keys", "equal keys", "equal rows, huge", "tiny", "one infinity"])
def test_selection_of_ties_everywhere(msa, what):
    """Every block undecided by fp32 (a dummy batch, one token over and over): the lower ids, and what differs by a bit."""
    import torch

    b = ref.Batch(counts=[1, 2], lens=[128 * 300 + 5, 128 * 41], Hq=2, G=2, seed=31)
    if what == "zero queries":
        b.q_idx[:] = 0
    elif what == "zero keys":
        b.k_idx[:] = 0
    elif what == "equal keys":
        b.k_idx[:] = torch.randn(64, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    elif what == "equal rows, huge":
        b.k_idx[:] = (torch.randn(64, generator=torch.Generator().manual_seed(3)) * 2.0 ** 70).to(torch.bfloat16)
        b.q_idx *= 2.0 ** 30
    elif what == "tiny":
        b.k_idx[:] = (torch.randn(64, generator=torch.Generator().manual_seed(3)) * 2.0 ** -70).to(torch.bfloat16)
    else:
        b.k_idx[:] = 1.0
        b.k_idx[int(b.table[0, 250]), 3, 7] = INF
        b.q_idx[:, :, 7] = b.q_idx[:, :, 7].abs() + 1
    if what != "zero keys":
        b.k_idx[int(b.table[1, 33]), 9] *= 1.5  # one key of one block
    O, LSE, bi = _sparse(msa, b, 16)
    for r in range(b.n):
        np.testing.assert_array_equal(bi[r], ref.select(b, r, 16))


@pytest.mark.parametrize("what", ["past 53 bits", "past 57 bits", "past 70 bits"])
def test_selection_of_one_key_in_many_places(msa, what):
    """A key that fills some blocks and stands once in others, with products too far apart for a sum in doubles to be
    exact: however a block's score is computed, it is the same everywhere, and the lower ids are taken."""
    import torch

    b = ref.Batch(counts=[1, 2], lens=[128 * 90 + 5, 128 * 41 + 77], Hq=2, G=2, seed=33)
    gen = torch.Generator().manual_seed(4)
    e = {"past 53 bits": 27, "past 57 bits": 28, "past 70 bits": 30}[what]
    for g in range(2):
        b.q_idx[:b.n, g] = 2.0 ** -e
        if e > 27:  # all of their bits
            b.q_idx[:b.n, g] = (2.0 ** -e * (1 + torch.rand(64, generator=gen))).to(torch.bfloat16)
    b.q_idx[:b.n, :, 0] = 1.0
    for s in range(2):
        key = (2.0 ** -e * (1 + (torch.rand(64, generator=gen) if e > 27 else torch.zeros(64)))).to(torch.bfloat16)
        key[0] = 1.0
        for c in range((b.lens[s] - 1) // 128):
            page = int(b.table[s, c])
            b.k_idx[page] = (torch.randn(128, 64, generator=gen) * 2.0 ** -e).to(torch.bfloat16)
            b.k_idx[page, :, 0] = 0.5
            b.k_idx[page, 77 if c % 3 == 0 else slice(None)] = key
    for k in (4, 9, 30):
        _, _, bi = _sparse(msa, b, k)
        for r in range(b.n):
            last = b.row_pos[r] // 128
            want = [*range(min(k - 1, last)), last]
            for g in range(2):
                assert bi[r, g].tolist()[:len(want)] == want, (r, g, k)


def test_dense_large_scores(msa):
    """Scores whose maximum moves by far more than exp2's range from page to page."""
    b = ref.Batch(counts=[2, 1, 1], lens=[128 * 6 + 90, 128 * 7, 128 * 6 + 1], Hq=8, G=2, prefix=4, seed=9)
    for s in range(3):
        for c in range(6):
            b.K[int(b.table[s, c])] *= 1.0 if s else float(1 + 3 * c)
    b.Q *= 4
    O, LSE = _dense(msa, b)
    ref.check_attention(b, range(b.n), range(b.Hq), O, LSE, _all(b), bf16_p=True)


def test_later_rows_do_not_reach_earlier_ones(msa):
    """Infinite and NaN values of a sequence's later rows: the rows before them are as without them."""
    b = ref.Batch(counts=[6, 5], lens=[262, 5], Hq=4, G=2, seed=10)
    clean = _dense(msa, b)
    for s in range(2):
        for i, v in ((1, NAN), (3, INF)):  # the sequence's last but i row
            t = b.lens[s] - 1 - i
            b.V[int(b.table[s, t // 128]), :, t % 128] = v
            b.K[int(b.table[s, t // 128]), :, t % 128] = v
    O, LSE = _dense(msa, b)
    for r in range(b.n):
        if b.row_pos[r] < b.lens[b.row_seq[r]] - 4:
            assert bool((O[r] == clean[0][r]).all()) and bool((LSE[r] == clean[1][r]).all()), r


# Batches of every path: single rows, rows that share a tile of eight columns, 128-row tiles (two of them, two groups),
# behind a prefix that is read as own pages, once for the batch, or in front of 128-row tiles.
PATHS = {
    "single": dict(counts=[1, 1], lens=[128 * 20 + 9, 300], Hq=16, G=2),
    "single_whole": dict(counts=[1] * 90, lens=[128 * 4 + 9 + i for i in range(90)], Hq=16, G=2),
    "columns": dict(counts=[3, 1, 4], lens=[128 * 6 + 9, 300, 128 * 2], Hq=2, G=1),
    "tiles": dict(counts=[20, 33], lens=[600, 128 * 9 + 40], Hq=16, G=2),
    "tiles_two_groups": dict(counts=[5, 9], lens=[600, 128 * 9 + 40], Hq=16, G=2),
    "folded": dict(counts=[1, 1, 1], lens=[128 * 6 + 9, 128 * 5 + 3, 128 * 7], Hq=8, G=2, prefix=5),
    "prefix": dict(counts=[1] * 20, lens=[128 * 40 + 3 + 9 * i for i in range(20)], Hq=8, G=2, prefix=40),
    "prefix_and_tiles": dict(counts=[3, 18], lens=[128 * 6 + 3, 128 * 6 + 400], Hq=16, G=2, prefix=6),
}


@pytest.mark.parametrize("name", PATHS)
def test_nan_scores_are_reported_as_such(msa, name):
    """A row whose visible scores are all NaN has LSE NaN (and not -infinity, which says that there was nothing to see),
    one that sees a single NaN as well; the other rows are as without them."""
    import torch

    b = ref.Batch(seed=22, **PATHS[name])
    clean = _dense(msa, b)
    rows, head = [0, b.n // 2], b.hg // 2  # a head of the first group
    for r in rows:
        b.Q[r, head] = NAN
    O, LSE = _dense(msa, b)
    bad = torch.zeros(b.n, b.Hq, dtype=torch.bool)
    bad[rows, head] = True
    assert bool(LSE[:b.n][bad].isnan().all()) and bool(O[:b.n][bad].isnan().all())
    assert torch.equal(LSE[:b.n][~bad], clean[1][:b.n][~bad]) and torch.equal(O[:b.n][~bad], clean[0][:b.n][~bad])
    # a block of NaN keys, of which a row has selected nothing but, or others too
    if not b.prefix:
        b = ref.Batch(seed=22, **PATHS[name])
        b.K[int(b.table[0, 1])] = NAN
        shape, cache, t = b.gpu(16)
        for ids in ([1], [0, 1], [1, 2], [0, 1, 2, 3]):
            bi = torch.full((b.N, b.G, 16), -1, dtype=torch.int32)
            bi[:, :, 0] = 0
            bi[0, 0, :len(ids)] = torch.tensor(ids)
            ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_SPARSE)
            O, LSE, _ = msa.paged_sparse_attn(shape, cache, t["Q"], block_idx=bi.cuda(), workspace=ws)
            msa.msa_check_device_status(ws)
            assert bool(LSE[0, :b.hg].isnan().all()) and bool(O[0, :b.hg].isnan().all()), ids
            assert not bool(LSE[0, b.hg:].isnan().any()) and not bool(LSE[1:b.n].isnan().any())


def _with_infinities(b, clean, blocks_of):
    """What rows are to have whose V holds infinities or NaN in some places: those (every visible token counts for more
    than 0), and `clean`, the result without them, elsewhere."""
    import torch

    want = clean.clone()
    for r in range(b.n):
        for g in range(b.G):
            blocks = [c for c in blocks_of(r, g) if c >= 0]
            v = b.V[b.table[b.row_seq[r], blocks].long(), g].reshape(-1, 128).float()
            token = (torch.tensor(blocks)[:, None] * 128 + torch.arange(128)).reshape(-1)
            odd = torch.where(v.isfinite(), 0.0, v)[token <= b.row_pos[r]].sum(0).to(torch.bfloat16)
            heads = slice(g * b.hg, (g + 1) * b.hg)
            want[r, heads] = torch.where(odd == 0, want[r, heads], odd)
    return want


@pytest.mark.parametrize("name", PATHS)
def test_infinite_values(msa, name):
    """An infinity in V, in the cache or among the new rows, gives that infinity wherever it is seen (both signs, or NaN:
    NaN), and changes nothing else. Some tokens have the row's largest score, whose probability is 1 before the sum."""
    import torch

    b = ref.Batch(seed=23, **PATHS[name])
    clean = _dense(msa, b)
    shape, cache, t = b.gpu(3)
    last = torch.tensor([p // 128 for p in b.row_pos])
    bi = torch.full((b.N, b.G, 3), -1, dtype=torch.int32)
    bi[:b.n, :, 0], bi[:b.n, :, 1] = 0, last[:, None]
    bi[:b.n][last == 0, :, 1] = -1
    sparse = (lambda r, g: bi[r, g].tolist())
    clean_s = msa.paged_sparse_attn(shape, cache, t["Q"], block_idx=bi.cuda())
    clean_s = [x[:b.n].cpu() for x in clean_s[:2]]
    rng = np.random.default_rng(1)
    for s in range(b.S):
        pages = b.table[s, :-(-b.lens[s] // 128)].tolist()
        for c, page in enumerate(pages):
            end = min(128, b.lens[s] - 128 * c)
            b.V[page, :, :end, 3] = INF             # every token, the one with the largest score among them
            b.V[page, :, rng.integers(end), 17] = -INF
            if c == len(pages) - 1:                 # among the new rows
                b.V[page, :, end - 1, 40] = INF
            if c == 0:
                b.V[page, :, 5, 64] = INF           # both signs
                b.V[page, :, 9, 64] = -INF
                b.V[page, :, 11, 90] = NAN
                b.V[page, 0, 127, 127] = INF
    O, LSE = _dense(msa, b)
    assert torch.equal(LSE[:b.n], clean[1][:b.n])
    want = _with_infinities(b, clean[0][:b.n], _all(b))
    assert torch.equal(O[:b.n].nan_to_num(nan=1e30, posinf=2e30, neginf=-2e30),
                       want.nan_to_num(nan=1e30, posinf=2e30, neginf=-2e30))
    assert int(want.isnan().sum()) and int((want == INF).sum()) and int((want == -INF).sum())
    t["V"].copy_(b.V)
    O, LSE, _ = msa.paged_sparse_attn(shape, cache, t["Q"], block_idx=bi.cuda())
    assert torch.equal(LSE[:b.n].cpu(), clean_s[1])
    want = _with_infinities(b, clean_s[0], sparse)
    assert torch.equal(O[:b.n].cpu().nan_to_num(nan=1e30, posinf=2e30, neginf=-2e30),
                       want.nan_to_num(nan=1e30, posinf=2e30, neginf=-2e30))


@pytest.mark.parametrize("name", [*PATHS, "one_long"])
def test_keys_that_nobody_attends_to(msa, name):
    """Scores of -infinity (an infinite key value) count for nothing: in the first page, on whole runs of pages, on the
    whole shared prefix, on every page but the row's own."""
    kw = PATHS.get(name) or dict(counts=[1], lens=[128 * 240 + 9], Hq=8, G=8, prefix=200)
    for which in ("first", "prefix", "all but the own"):
        b = ref.Batch(seed=24, **kw)
        assert min(b.row_pos) >= 128
        b.Q[:, :, 0] = 1.0
        own = [min(p for p, s in zip(b.row_pos, b.row_seq) if s == i) // 128 for i in range(b.S)]  # of the first row
        n = {"first": [1] * b.S, "prefix": [max(1, b.prefix)] * b.S, "all but the own": own}[which]
        for s in range(b.S):
            for c in range(n[s]):
                b.K[int(b.table[s, c]), :, :, 0] = -INF
        # (in a page that is shared, all the tokens)
        O, LSE = _dense(msa, b)
        rows = range(b.n) if b.n < 30 else range(0, b.n, 7)
        ref.check_attention(b, rows, range(0, b.Hq, 3), O, LSE,
                            lambda r, g: list(range(n[b.row_seq[r]], b.row_pos[r] // 128 + 1)), bf16_p=b.prefix > 5)


def _slots(msa, shape):
    """Parts of a row's output that the full call's workspace has room for."""
    return msa.msa_paged_workspace_size(shape, msa.MSA_WS_PAGED_DENSE) // (shape.N * shape.Hq * 516)


def _rising(b, pages, step=0.8, again=40):
    """Scores that grow from page to page, by turns those of a page's first half, of its second one, and of all its keys."""
    for i, page in enumerate(pages):
        f = 1 + step * (i % again)
        b.K[page, :, :64] *= f if i % 3 != 1 else 0.25
        b.K[page, :, 64:] *= f if i % 3 != 0 else 0.25


# Prefixes whose runs of pages are long: over more pages than are looked up at a time, and from one group to the next.
LONG = {
    "g3_hg8": dict(S=340, rows=1, blocks=203, Hq=24, G=3, prefix=201),
    "g7_hg4": dict(S=300, rows=2, blocks=101, Hq=28, G=7, prefix=100),
    "g2_hg1": dict(S=1500, rows=1, blocks=402, Hq=2, G=2, prefix=401),
    "tiles_g8_hg2": dict(S=200, rows=5, blocks=106, Hq=16, G=8, prefix=100),
    "tiles_g5_hg8": dict(S=30, rows=19, blocks=153, Hq=40, G=5, prefix=150),
}


@pytest.mark.parametrize("rising", [False, True], ids=["even", "rising"])
@pytest.mark.parametrize("name", LONG)
def test_dense_prefix_long_runs(msa, name, rising):
    kw = dict(LONG[name])
    prefix, blocks = kw.pop("prefix"), kw.pop("blocks")
    b = _shared_pages(length=128 * blocks - 70, seed=41, **kw)
    b.prefix = prefix
    if rising:
        _rising(b, b.table[0, :prefix].tolist())
    shape, _, _ = b.gpu()
    before = msa.msa_kernel_launches()
    O, LSE = _dense(msa, b)
    assert msa.msa_kernel_launches() - before == (3 if name.startswith("tiles") else 4)
    # parts of a row: the prefix's and at least one of its own pages
    assert prefix / (_slots(msa, shape) - 1) > 20
    rows = sorted({0, 1, 15, 16, 17, b.n // 2, b.n - 1})
    ref.check_attention(b, rows, range(0, b.Hq, 5 if b.Hq > 8 else 1), O, LSE, _all(b), bf16_p=True)


@pytest.mark.parametrize("S,rows,blocks,Hq,G", [(90, 5, 12, 16, 8), (60, 70, 11, 16, 8), (160, 9, 10, 24, 3), (170, 3, 40, 8, 1)],
                         ids=["twin", "two_tiles", "one_tile", "one_group"])
def test_dense_rows_rising_scores(msa, S, rows, blocks, Hq, G):
    """Runs of several own pages whose maxima rise, in both halves of a page and in either."""
    b = _shared_pages(S, rows, 128 * blocks - 70, Hq, G, seed=43)
    _rising(b, b.table[0, :blocks].tolist(), again=blocks)
    shape, _, _ = b.gpu()
    before = msa.msa_kernel_launches()
    O, LSE = _dense(msa, b)
    assert msa.msa_kernel_launches() - before == 3
    assert blocks / _slots(msa, shape) >= 4
    some = sorted({0, 1, rows - 1, rows, b.n // 2, b.n - 1})
    ref.check_attention(b, some, range(0, Hq, 3), O, LSE, _all(b))


@pytest.mark.parametrize("name", ["prefix1", "prefix_hg1", "prefix_hg2", "prefix_hg4_rows", "prefix_idle_first",
                                  "large scores"])
def test_dense_prefix_read_as_own_pages(msa, name):
    """Behind a small shared prefix the probabilities have 16 bits, as without one."""
    if name == "large scores":
        b = ref.Batch(counts=[2, 1, 1], lens=[128 * 6 + 90, 128 * 7, 128 * 6 + 1], Hq=8, G=2, prefix=4, seed=9)
        for s in range(3):
            for c in range(6):
                b.K[int(b.table[s, c])] *= 1.0 if s else float(1 + 3 * c)
        b.Q *= 4
    else:
        b = ref.Batch(seed=6, **DENSE[name])
    before = msa.msa_kernel_launches()
    O, LSE = _dense(msa, b)
    assert msa.msa_kernel_launches() - before == 2  # rows and attention
    heads = range(b.Hq) if b.Hq <= 8 else range(0, b.Hq, 5)
    ref.check_attention(b, range(0, b.n, 1 if b.n < 30 else 7), heads, O, LSE, _all(b))


@pytest.mark.parametrize("rows,Hq,launches", [(1, 8, 4), (20, 64, 3)], ids=["shared", "tiles"])
def test_prefix_in_pools_past_32_bit_offsets(msa, rows, Hq, launches):
    """A shared prefix (and own pages of 128-row tiles) more than 2^31 elements into the pools."""
    import torch

    G, pages = 8, 17000
    K, V = (torch.zeros(pages, G, 128, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    b = ref.Batch(counts=[rows], lens=[128 * 192 + 30], Hq=Hq, G=G, prefix=190, seed=13, spare=0, index=False)
    far = torch.tensor([pages - 1 - 2 * i for i in range(b.num_pages)], device="cuda")
    assert int(far.min()) * G * 128 * 128 > 2 ** 31
    K[far], V[far] = b.K.cuda(), b.V.cuda()
    table = far.cpu()[b.table.long()].to(torch.int32).cuda()
    cache = msa.PagedCache(K, V, None, table, torch.tensor([0, rows], dtype=torch.int32, device="cuda"),
                           torch.tensor(b.lens, dtype=torch.int32, device="cuda"))
    shape = msa.PagedShape(S=1, N=rows, Hq=Hq, G=G, num_pages=pages, max_blocks=b.max_blocks, prefix_blocks=190)
    before = msa.msa_kernel_launches()
    O, LSE = msa.paged_dense_attn(shape, cache, b.Q.cuda())
    assert msa.msa_kernel_launches() - before == launches
    ref.check_attention(b, range(0, rows, 6), range(0, Hq, 5), O.cpu(), LSE.cpu(), _all(b), bf16_p=True)
    del K, V


def test_pools_past_32_bit_offsets(msa):
    """Pages whose values lie more than 2^31 elements (and 2^32 bytes) into the pools."""
    import torch

    G, pages = 8, 16500
    K, V = (torch.zeros(pages, G, 128, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k_idx = torch.zeros(pages, 128, 64, dtype=torch.bfloat16, device="cuda")
    b = ref.Batch(counts=[1], lens=[128 * 9 + 30], Hq=8, G=G, seed=13, spare=0)
    far = torch.tensor([pages - 1 - 3 * i for i in range(b.num_pages)], device="cuda")
    K[far], V[far], k_idx[far] = b.K.cuda(), b.V.cuda(), b.k_idx.cuda()
    table = far.cpu()[b.table.long()].to(torch.int32).cuda()
    one, ln = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor(b.lens, dtype=torch.int32, device="cuda")
    cache = msa.PagedCache(K, V, k_idx, table, one, ln)
    shape = msa.PagedShape(S=1, N=1, Hq=8, G=G, num_pages=pages, max_blocks=b.max_blocks, k=5)
    O, LSE, bi = msa.paged_sparse_attn(shape, cache, b.Q.cuda(), b.q_idx.cuda())
    np.testing.assert_array_equal(bi[0].cpu().numpy(), ref.select(b, 0, 5))
    ref.check_attention(b, [0], range(8), O.cpu(), LSE.cpu(), lambda r, g: bi[r, g].tolist())
    shape4 = msa.PagedShape(S=1, N=1, Hq=8, G=G, num_pages=pages, max_blocks=b.max_blocks, prefix_blocks=4)
    O, LSE = msa.paged_dense_attn(shape4, cache, b.Q.cuda())
    ref.check_attention(b, [0], range(8), O.cpu(), LSE.cpu(), _all(b), bf16_p=True)
    new = torch.randn(1, G, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    msa.paged_append(shape, cache, msa.Rope(), new, new)
    assert torch.equal(K[int(far[b.table[0, 9].long()]), :, 29], new[0])
    del K, V, k_idx


# ----------------------------------------------------------------- the batch description's faults
def test_bad_pages_and_positions_are_reported(msa):
    import torch

    def run(change, which="sparse", prefix=0, good=None):
        b = ref.Batch(counts=[1, 2], lens=[128 * 5 + 3, 128 * 6 + 9], Hq=8, G=2, prefix=prefix, seed=1)
        change(b)
        shape, cache, t = b.gpu(4)
        if which == "append":
            ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_APPEND)
            new = torch.ones(b.N, 2, 128, dtype=torch.bfloat16, device="cuda")
            msa.paged_append(shape, cache, msa.Rope(), new, new, workspace=ws)
        elif which == "sparse":
            ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_SPARSE)
            O, LSE, bi = msa.paged_sparse_attn(shape, cache, t["Q"], t["q_idx"], workspace=ws)
        else:
            ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_DENSE)
            O, LSE = msa.paged_dense_attn(shape, cache, t["Q"], workspace=ws)
        with pytest.raises(msa.MsaError) as e:
            msa.msa_check_device_status(ws)
        assert e.value.status == msa.MSA_ERR_DEVICE
        msa.msa_check_device_status(ws)  # the word was cleared
        if good is not None:  # the rows that were in order
            blocks = (lambda r, g: bi[r, g].tolist()) if which == "sparse" else _all(b)
            ref.check_attention(b, good, range(8), O.cpu(), LSE.cpu(), blocks, bf16_p=prefix > 0)

    def page(s, c, v):
        def change(b):
            b.table[s, c] = v
        return change

    def length(s, v):
        def change(b):
            b.lens[s] = v
        return change

    for v in (-1, 1 << 20, 2 ** 31 - 1, -2 ** 31):
        run(page(0, 2, v), "sparse", good=[1, 2])
        run(page(1, 6, v), "sparse", good=[0])
        run(page(0, 5, v), "dense", good=[1, 2])
        run(page(0, 5, v), "append")
        run(page(0, 1, v), "dense", prefix=3)
    for v in (0, -5, 128 * 7 + 1, 2 ** 31 - 1, -2 ** 31):
        run(length(0, v), "sparse", good=[1, 2])
        run(length(0, v), "dense", good=[1, 2])
        run(length(0, v), "append")
    run(length(1, 128 * 3 + 1), "dense", prefix=3, good=[0])  # a row inside the prefix
    run(page(1, 2, 0), "dense", prefix=3)                      # a prefix that is not shared


def test_bad_selections_are_reported(msa):
    import torch

    for ids in ([0, 6, -1], [3, 1, 5], [2, 2, 5], [0, -1, 5], [-5, 1, 2], [2 ** 31 - 1, -1, -1]):
        b = ref.Batch(counts=[1, 1], lens=[128 * 5 + 3, 128 * 5 + 3], Hq=8, G=2, seed=1)
        bi = torch.tensor([[[0, 2, 5]] * 2] * 2, dtype=torch.int32)
        bi[0, 1] = torch.tensor(ids, dtype=torch.int32)
        shape, cache, t = b.gpu(3)
        ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_SPARSE)
        O, LSE, _ = msa.paged_sparse_attn(shape, cache, t["Q"], block_idx=bi.cuda(), workspace=ws)
        with pytest.raises(msa.MsaError) as e:
            msa.msa_check_device_status(ws)
        assert e.value.status == msa.MSA_ERR_DEVICE, ids
        ref.check_attention(b, [1], range(8), O.cpu(), LSE.cpu(), lambda r, g: [0, 2, 5])


@pytest.mark.parametrize("S,G", [(2, 2), (40, 8)], ids=str)  # a row's list cut into several parts, and not cut
@pytest.mark.parametrize("k,ids", [(8, [0] * 8), (8, [0, 1, 2, 3, 3, 3, 3, 3]), (6, [0, 1, 2, 3, 4, 5]), (128, [3] * 128),
                                   (128, list(range(128))), (9, [0, 1, 2, 3] + [2 ** 31 - 1] * 5)],
                         ids=["zeros", "one_again", "past_the_table", "equal_128", "all_128", "huge"])
def test_selections_longer_than_the_page_table_are_reported(msa, S, G, k, ids):
    """More ids than the table has columns (k may be larger): no part of a row is counted that has no place in the
    workspace, and the other rows are as they should be."""
    import torch

    b = ref.Batch(counts=[1] * S, lens=[128 * 3 + 5 + i for i in range(S)], Hq=G, G=G, seed=1)
    assert b.max_blocks == 4
    bi = torch.full((S, G, k), -1, dtype=torch.int32)
    bi[:, :, :3] = torch.tensor([0, 2, 3])
    good = bi.clone()
    bi[0, 1] = torch.tensor(ids, dtype=torch.int32)
    if S > 2:
        bi[S // 2, 0] = torch.tensor(ids, dtype=torch.int32)
    shape, cache, t = b.gpu(k)
    ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_SPARSE)
    for fill in (0, 255, 1):  # (what a count of parts might be taken for)
        ws.fill_(fill)
        O, LSE, _ = msa.paged_sparse_attn(shape, cache, t["Q"], block_idx=bi.cuda(), workspace=ws)
        with pytest.raises(msa.MsaError) as e:
            msa.msa_check_device_status(ws)
        assert e.value.status == msa.MSA_ERR_DEVICE
        ref.check_attention(b, [1, S - 1], range(G), O.cpu(), LSE.cpu(), lambda r, g: [0, 2, 3])
        O, LSE, _ = msa.paged_sparse_attn(shape, cache, t["Q"], block_idx=good.cuda(), workspace=ws)
        msa.msa_check_device_status(ws)
        ref.check_attention(b, [0, S - 1], range(G), O.cpu(), LSE.cpu(), lambda r, g: [0, 2, 3])


# ----------------------------------------------------------------- streams, graphs, reruns
def test_copied_cache_has_its_own_tensors(msa):
    """A deep copy is another cache: appending to it leaves the first one alone, and works after that one is gone."""
    import copy

    import torch

    b = ref.Batch(counts=[1, 3], lens=[130, 259], Hq=8, G=2, seed=7, stale=0.0)
    shape, cache, t = b.gpu()
    same, other = copy.copy(cache), copy.deepcopy(cache)
    assert same.K.data_ptr() == cache.K.data_ptr() and other.K.data_ptr() != cache.K.data_ptr()
    assert other._struct.K == other.K.data_ptr() and other._struct.seq_len == other.seq_len.data_ptr()
    before = t["K"].clone()
    new = torch.ones(b.N, 2, 128, dtype=torch.bfloat16, device="cuda")
    msa.paged_append(shape, other, msa.Rope(), new, new)
    assert torch.equal(cache.K, before) and not torch.equal(other.K, before)
    msa.paged_append(shape, same, msa.Rope(), new, new)
    assert torch.equal(cache.K, other.K)


def test_same_bits_on_other_streams_and_at_once(msa):
    import torch

    b = ref.Batch(counts=[1, 4, 2], lens=[3000, 2500, 1200], Hq=16, G=4, seed=2)
    p = ref.Batch(counts=[1] * 9, lens=[128 * 30 + 5 + i for i in range(9)], Hq=16, G=4, prefix=30, seed=2)
    O, LSE, bi = _sparse(msa, b, 8)
    Od, LSEd = _dense(msa, p)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    s1.wait_stream(torch.cuda.current_stream())
    s2.wait_stream(torch.cuda.current_stream())
    kept = []
    for _ in range(3):
        with torch.cuda.stream(s1):
            shape, cache, t = b.gpu(8)
            kept.append((cache, t) + msa.paged_sparse_attn(shape, cache, t["Q"], t["q_idx"]))
        shape, cache, t = p.gpu()
        s2.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s2):
            ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_DENSE)
        kept.append((cache, t, ws) + msa.paged_dense_attn(shape, cache, t["Q"], workspace=ws, stream=s2))
    torch.cuda.synchronize()
    for i in range(0, 6, 2):
        assert torch.equal(kept[i][2].cpu(), O) and torch.equal(kept[i][3].cpu(), LSE)
        np.testing.assert_array_equal(kept[i][4].cpu().numpy(), bi)
        assert torch.equal(kept[i + 1][3].cpu(), Od) and torch.equal(kept[i + 1][4].cpu(), LSEd)


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_helpers_allocate_on_the_stream_they_run_on(msa, raw):
    """A helper on a side stream without a workspace: what it allocates is neither handed out to the current stream while
    the side stream still has the call to do, nor taken from what the current stream still writes to."""
    import torch

    b = ref.Batch(counts=[1, 2], lens=[128 * 30 + 4, 128 * 25], Hq=8, G=2, seed=17, stale=0.0)
    shape, cache, t = b.gpu(6)
    want_s = [x.clone() for x in msa.paged_sparse_attn(shape, cache, t["Q"], t["q_idx"])]
    want_d = [x.clone() for x in msa.paged_dense_attn(shape, cache, t["Q"])]
    new = torch.zeros(b.N, 2, 128, dtype=torch.bfloat16, device="cuda")
    scratch = ref.Batch(counts=[1, 2], lens=[128 * 30 + 4, 128 * 25], Hq=8, G=2, seed=18, stale=0.0).gpu(6)[1]
    want_q, _ = msa.paged_append(shape, scratch, msa.Rope(_freq(128).cuda()), new, new, Q=t["Q"])
    want_q = want_q.clone()
    rope = msa.Rope(_freq(128).cuda())
    sizes = [msa.msa_paged_workspace_size(shape, w) for w in range(3)]
    sizes += [x.nbytes for x in want_s + want_d + [want_q]]
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    stream = side.cuda_stream if raw else side
    torch.cuda.synchronize()
    for _ in range(10):
        # the current stream is busy with memory that it has given back
        torch.cuda._sleep(3_000_000)
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_000_000)
        s = msa.paged_sparse_attn(shape, cache, t["Q"], t["q_idx"], stream=stream)
        d = msa.paged_dense_attn(shape, cache, t["Q"], stream=stream)
        q, _ = msa.paged_append(shape, scratch, rope, new, new, Q=t["Q"], stream=stream)
        # and takes memory while the side stream has not come to the calls
        held = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) for n in sizes * 2]
        here.wait_stream(side)
        for got, want in list(zip(s, want_s)) + list(zip(d, want_d)) + [(q, want_q)]:
            assert torch.equal(got, want)
        del s, d, q, got, held


def test_captured_step_replays_on_another_batch(msa):
    """One decode step (append, selection and attention, full attention) captured once, replayed with other lengths,
    pages and rows of the same shape; two graphs share nothing but the cache."""
    import torch

    b = ref.Batch(counts=[1, 2, 1], lens=[900, 700, 129], Hq=8, G=2, pad=2, seed=20, max_blocks=12, spare=8, stale=0.0)
    shape, cache, t = b.gpu(4)
    N = b.N
    new = {n: torch.zeros(N, *s, dtype=torch.bfloat16, device="cuda")
           for n, s in (("K", (2, 128)), ("V", (2, 128)), ("k_idx", (64,)), ("Q", (8, 128)), ("q_idx", (2, 64)))}
    rope = msa.Rope(_freq(128).cuda(), _freq(64).cuda())
    wsa, wss, wsd = (msa.alloc_paged_workspace(shape, w) for w in range(3))
    Qr, qir = torch.zeros_like(new["Q"]), torch.zeros_like(new["q_idx"])
    O, Od = torch.zeros_like(Qr), torch.zeros_like(Qr)
    LSE, LSEd = (torch.zeros(N, 8, device="cuda") for _ in range(2))
    bi = torch.zeros(N, 2, 4, dtype=torch.int32, device="cuda")

    def step():
        msa.msa_paged_append(shape, cache, rope, new["K"], new["V"], new["k_idx"], new["Q"], new["q_idx"], Qr, qir, wsa)
        msa.msa_paged_sparse_attn(shape, cache, Qr, qir, bi, O, LSE, wss)
        msa.msa_paged_dense_attn(shape, cache, Qr, Od, LSEd, wsd)

    step()  # once before the capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed, counts, lens in ((1, [1, 2, 1], [900, 700, 129]), (2, [0, 1, 4], [0, 1300, 500]), (3, [6, 0, 0], [6, 0, 0])):
        c = ref.Batch(counts=counts, lens=lens, Hq=8, G=2, pad=N - sum(counts), seed=seed, max_blocks=12, spare=0,
                      stale=0.0)
        gen = torch.Generator().manual_seed(seed)
        t["table"].copy_(c.table)
        t["row_start"].copy_(torch.tensor(c.starts, dtype=torch.int32))
        t["seq_len"].copy_(torch.tensor(lens, dtype=torch.int32))
        for n in ("K", "V", "k_idx"):
            t[n].zero_()
            t[n][:c.num_pages].copy_(getattr(c, n))
        for v in new.values():
            v.copy_(torch.randn(v.shape, generator=gen))
        g.replay()
        for ws in (wsa, wss, wsd):
            msa.msa_check_device_status(ws)
        c.K, c.V, c.k_idx = (t[n].cpu() for n in ("K", "V", "k_idx"))
        c.Q, c.q_idx = Qr.cpu(), qir.cpu()
        got = bi.cpu().numpy()
        for r in range(c.n):
            np.testing.assert_array_equal(got[r], ref.select(c, r, 4))
        ref.check_attention(c, range(c.n), range(8), O.cpu(), LSE.cpu(), lambda r, g_: got[r, g_].tolist())
        ref.check_attention(c, range(c.n), range(8), Od.cpu(), LSEd.cpu(), _all(c))


# ----------------------------------------------------------------- together, as a model would use them
def test_served_rows_are_those_of_the_training_calls(msa):
    """A sequence written into the cache in pieces (a prompt, drafts, single tokens) and attended to from there gives
    what msa_index_topk + msa_sparse_fwd and msa_dense_fwd give for the whole sequence at once."""
    import torch

    T, Hq, G, k = 1536, 8, 2, 5
    gen = torch.Generator().manual_seed(30)

    def normal(*shape):
        return torch.randn(*shape, generator=gen).to(torch.bfloat16).cuda()

    Q, K, V, qi, ki = normal(T, Hq, 128), normal(T, G, 128), normal(T, G, 128), normal(T, G, 64), normal(T, 64)
    f, fi = _freq(128).cuda(), _freq(64).cuda()
    pages = 20
    order = torch.randperm(pages, generator=gen)[:12].to(torch.int32)
    pk, pv = (torch.full((pages, G, 128, 128), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pi = torch.full((pages, 128, 64), NAN, dtype=torch.bfloat16, device="cuda")
    table = order.view(1, 12).cuda()
    got = {n: [] for n in ("Q", "qi", "O", "LSE", "bi", "Od", "LSEd")}
    at = 0
    for n in (700, 1, 1, 5, 128, 61, 512, 1, 127):
        cache = msa.PagedCache(pk, pv, pi, table, torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                               torch.tensor([at + n], dtype=torch.int32, device="cuda"))
        shape = msa.PagedShape(S=1, N=n, Hq=Hq, G=G, num_pages=pages, max_blocks=12, k=k, prefix_blocks=at // 128)
        s = slice(at, at + n)
        Qr, qir = msa.paged_append(shape, cache, msa.Rope(f, fi), K[s], V[s], ki[s], Q[s], qi[s])
        O, LSE, bi = msa.paged_sparse_attn(shape, cache, Qr, qir)
        Od, LSEd = msa.paged_dense_attn(shape, cache, Qr)  # the sequence's own full blocks as the shared prefix
        for name, v in zip(got, (Qr, qir, O, LSE, bi, Od, LSEd)):
            got[name].append(v)
        at += n
    assert at == T
    got = {n: torch.cat(v) for n, v in got.items()}
    # the rotated sequence, read back from the pages
    Kr = pk[order.long().cuda()].transpose(1, 2).reshape(1, T, G, 128).contiguous()
    Vr = pv[order.long().cuda()].transpose(1, 2).reshape(1, T, G, 128).contiguous()
    kir = pi[order.long().cuda()].reshape(1, T, 64).contiguous()
    assert torch.equal(Vr[0], V)
    s = msa.Shape(B=1, T=T, Hq=Hq, G=G, k=k)
    bi = msa.index_topk(s, got["qi"][None].contiguous(), kir)
    same = (bi[0].transpose(0, 1) == got["bi"]).all(dim=2)
    assert float(same.float().mean()) > 0.999  # the training call decides near-ties in fp32
    O, LSE = msa.sparse_fwd(s, got["Q"][None].contiguous(), Kr, Vr, bi)
    Od, LSEd = msa.dense_fwd(s, got["Q"][None].contiguous(), Kr, Vr)
    same = same.repeat_interleave(Hq // G, dim=1)
    # both round P to bf16 at most, O to bf16, from scores within 1e-4: 2^-8 of |O| twice and of sum p |v| (< 4.5) once
    for a, c, m in ((got["O"], O[0], same), (got["Od"], Od[0], torch.ones_like(same))):
        err = (a.float() - c.float()).abs()
        assert float((err * m[..., None]).max()) <= 2.0 ** -8 * (4.5 + 2 * float(c.float().abs().max()))
        assert float((err * m[..., None]).mean()) <= 2.0 ** -8
    assert float(((got["LSE"] - LSE[0]).abs() * same).max()) <= 1e-3
    assert float((got["LSEd"] - LSEd[0]).abs().max()) <= 1e-3

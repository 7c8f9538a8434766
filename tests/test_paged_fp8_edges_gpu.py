"""Calls over a paged cache in 8 bits at the edges of what they take, on the GPU against their 64-bit forms (tests/paged_ref.py
and tests/paged_fp8_ref.py, bounds derived there)."""
import numpy as np
import pytest

import paged_fp8_ref as ref8
import paged_ref as ref
from test_paged_fp8_gpu import (DENSE, SCALES, SPARSE, TILES, _all, _check_padding, _check_sparse, _dense, _sparse,  # noqa: F401
                                msa)
from test_paged_gpu import _dense as _dense16

pytestmark = pytest.mark.gpu

INF = float("inf")


# ----------------------------------------------------------------- reading back
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("start,count", [(5, [10]), (31, [1, 0, 200]), (40, [0, 0, 129]), (2500, [300, 7, 130]), (3, [0, 0, 0])],
                         ids=str)
def test_read_leaves_the_rows_before_the_first_sequence_alone(msa, start, count, first):  # noqa: F811
    """A slice of a longer batch's starts: rows out_start[s] .. out_start[s + 1] - 1 are sequence s's, others nobody's."""
    import torch

    lens = [400, 150, 333][:len(count)]
    b = ref8.Batch(counts=[0] * len(lens), lens=lens, Hq=2, G=2, seed=2)
    shape, cache, t = b.gpu()
    starts = start + np.concatenate([[0], np.cumsum(count)])
    n = int(starts[-1])
    K, V = (torch.full((n + 3, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ki = torch.full((n + 3, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_APPEND)
    ws.fill_(255)
    at = [100, 20, 60][:len(count)] if first else [0] * len(count)
    msa.msa_paged_read_fp8(shape, cache, torch.tensor(at, dtype=torch.int32, device="cuda") if first else None,
                           torch.tensor(starts, dtype=torch.int32, device="cuda"), K, V, ki, ws)
    msa.msa_check_device_status(ws)
    for x in (K, V, ki):
        assert bool((x[:start] == 5.0).all()) and bool((x[n:] == 5.0).all())
    for s, c in enumerate(count):
        rows = slice(int(starts[s]), int(starts[s + 1]))
        token = torch.arange(c) + at[s]
        page, slot = b.table[s, token // 128].long(), token % 128
        assert torch.equal(K[rows].cpu(), b.K[page, :, slot]) and torch.equal(V[rows].cpu(), b.V[page, :, slot])
        assert torch.equal(ki[rows].cpu(), b.k_idx[page, slot])


# ----------------------------------------------------------------- scores
@pytest.mark.parametrize("up,down", [(90, -90), (112, -98), (118, -103), (-90, 90), (-114, 114)])
@pytest.mark.parametrize("name", SCALES)
def test_scores_of_far_powers_of_two(msa, name, up, down):  # noqa: F811
    """Keys of 2^up and queries of 2^down: their scores fit, whatever is multiplied first. One head's queries are smaller."""
    def change(b):
        b.K *= 2.0 ** up
        b.Q *= 2.0 ** down
        b.Q[:, 1] *= 2.0 ** -3

    b = ref8.Batch(seed=7, change=change, **SCALES[name])
    O, LSE = _dense(msa, b)
    assert bool(LSE[:b.n].isfinite().all()) and bool(O[:b.n].isfinite().all())
    rows = range(b.n) if b.n < 30 else range(0, b.n, 7)
    ref8.check_attention(b, rows, range(0, b.Hq, 1 if b.Hq <= 8 else 5), O, LSE, _all(b), bf16_p=ref8.tiles(b))
    _check_padding(b, O, LSE)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("name", SCALES)
def test_infinite_queries(msa, name, bits):  # noqa: F811
    """Every score of such a head is an infinity: with all of them negative the row sees nothing (O = 0, LSE = -infinity), one
    positive makes it NaN; keys far below 1 change nothing of that, and the other heads of the rows have the same bits."""
    import torch

    dense = _dense if bits == 8 else _dense16

    def change(b):
        b.K *= 2.0 ** -60
        b.K[..., 5] = b.K[..., 5].abs() + 2.0 ** -61

    if bits == 8:
        b = ref8.Batch(seed=8, change=change, **SCALES[name])
    else:
        b = ref.Batch(seed=8, **SCALES[name])
        change(b)
    clean = dense(msa, b)
    r = b.n - 1
    page, slot = int(b.table[b.row_seq[r], b.row_pos[r] // 128]), b.row_pos[r] % 128
    b.Q[r, 0] = 0.0
    b.Q[r, 0, 5] = -INF
    O, LSE = dense(msa, b)
    assert bool((O[r, 0] == 0).all()) and float(LSE[r, 0]) == -INF
    assert torch.equal(O[r, 1:], clean[0][r, 1:]) and torch.equal(O[:r], clean[0][:r]) and torch.equal(LSE[:r], clean[1][:r])
    # the row's own token: its score is +infinity
    if bits == 8:
        b.K8.view(torch.uint8)[page, 0, slot, 5] |= 128
    else:
        b.K[page, 0, slot, 5] *= -1
    O, LSE = dense(msa, b)
    assert bool(O[r, 0].isnan().all()) and not bool(O[r, b.hg:].isnan().any())

# ----------------------------------------------------------------- the largest magnitudes
@pytest.mark.parametrize("name", [*SCALES, *TILES])
def test_codes_past_the_largest_number_reach_their_rows_alone(msa, name):  # noqa: F811
    """The last token's V has a value that the format rounds to 2^128. The rows that see it may have any value in its dim;
    everything else has the same bits as with a zero there."""
    import torch

    kw = {**SCALES, **TILES}[name]
    b = ref8.Batch(seed=10, **kw)

    def put(code, d):
        for s in range(b.S):
            t = b.lens[s] - 1
            if b.counts[s]:
                at = (int(b.table[s, t // 128]), slice(None), t % 128)
                b.V_exp[at] = 247
                b.V8.view(torch.uint8)[at] = 0
                b.V8.view(torch.uint8)[(*at, d)] = code

    put(0, 0)
    clean = _dense(msa, b)
    for code, d in ((0x78, 3), (0xfe, 77), (0x7b, 126)):
        put(code, d)
        O, LSE = _dense(msa, b)
        assert torch.equal(LSE[:b.n], clean[1][:b.n])
        other = torch.arange(128) != d
        for r in range(b.n):
            if b.row_pos[r] == b.lens[b.row_seq[r]] - 1:
                assert torch.equal(O[r][:, other], clean[0][r][:, other]), r
            else:
                assert torch.equal(O[r], clean[0][r]), r


def test_append_and_read_of_the_largest_magnitudes(msa):  # noqa: F811
    """Up to where a code of 2^120 rounds to 256 a value comes back within 2^-4 of itself; from there on as an infinity."""
    import torch

    top = torch.arange(0x7f00, 0x7f80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)  # 2^127 and more
    x = torch.stack([top, -top])[:, None]
    b = ref8.Batch(counts=[2], lens=[2], Hq=1, G=1)
    shape, cache, t = b.gpu()
    msa.paged_append_fp8(shape, cache, msa.Rope(), x.cuda(), x.cuda(), x[:, 0, :64].contiguous().cuda())
    K, V, _ = msa.paged_read_fp8(shape, cache, torch.tensor([0, 2], dtype=torch.int32, device="cuda"), 2)
    for got in (K.cpu().double(), V.cpu().double()):
        y = x.double()
        fits = y.abs() < 248 * 2.0 ** 120
        assert bool(((got - y).abs() <= 2.0 ** -4 * y.abs())[fits].all())
        assert bool((got[~fits] == y[~fits].sign() * INF).all()) and int((~fits).sum()) == 2 * 8


# ----------------------------------------------------------------- probabilities
@pytest.mark.parametrize("name", [*DENSE, *SCALES])
def test_probabilities_by_eight_columns_have_eleven_bits(msa, name):  # noqa: F811
    """Two launches: eight columns at a time, whatever the batch's shape, also where they read a small shared prefix."""
    b = ref8.Batch(seed=6, **{**DENSE, **SCALES}[name])
    before = msa.msa_kernel_launches()
    O, LSE = _dense(msa, b)
    if msa.msa_kernel_launches() - before > 2:
        assert b.prefix or b.N * b.hg > 20 * b.S
        pytest.skip("128-row tiles")
    rows = range(b.n) if b.n < 30 else range(0, b.n, 7)
    ref8.check_attention(b, rows, range(0, b.Hq, 1 if b.Hq <= 8 else 5), O, LSE, _all(b))
    _check_padding(b, O, LSE)


@pytest.mark.parametrize("rows", [2, 3])
def test_up_to_twenty_columns_a_sequence_have_eleven_bits(msa, rows):  # noqa: F811
    """Without a prefix 128-row tiles take batches of more than 20 columns (rows x heads of a group) a sequence alone."""
    b = ref8.Batch(counts=[rows] * 20, lens=[1100 + 7 * i for i in range(20)], Hq=64, G=8, seed=6)
    before = msa.msa_kernel_launches()
    O, LSE = _dense(msa, b)
    assert msa.msa_kernel_launches() - before == (2 if rows == 2 else 3)
    ref8.check_attention(b, range(0, b.n, 7), range(0, 64, 5), O, LSE, _all(b), bf16_p=rows == 3)


# ----------------------------------------------------------------- tables as wide as a serving program's
@pytest.mark.parametrize("width", [200, 8192])
@pytest.mark.parametrize("name", ["rows_hg2_idle", "g8_long", "runs_hg8", "tokens", "shared", "prefix", "hg8_one_tile", "drafts",
                                  "two_rows"])
def test_dense_over_wide_tables(msa, name, width):  # noqa: F811
    """Columns past the sequences' ends (-1) change the cuts and nothing else."""
    b = ref8.Batch(seed=6, max_blocks=width, **{**DENSE, **SCALES, **TILES}[name])
    O, LSE = _dense(msa, b)
    rows = range(b.n) if b.n < 30 else range(0, b.n, 7)
    ref8.check_attention(b, rows, range(0, b.Hq, 1 if b.Hq <= 8 else 5), O, LSE, _all(b), bf16_p=ref8.tiles(b))
    _check_padding(b, O, LSE)


@pytest.mark.parametrize("width", [200, 8192])
@pytest.mark.parametrize("name", ["first_token", "hg2_idle_padding", "hg8_rows", "many_rows"])
def test_sparse_over_wide_tables(msa, name, width):  # noqa: F811
    kw = dict(SPARSE[name])
    k = kw.pop("k")
    b = ref8.Batch(seed=3, max_blocks=width, **kw)
    _check_sparse(b, k, *_sparse(msa, b, k))

"""Calls over a paged cache in 8 bits at the edges of what they take, on the GPU against their 64-bit forms (tests/paged_ref.py
and tests/paged_fp8_ref.py, bounds derived there)."""
import math

import numpy as np
import pytest

import paged_fp8_ref as ref8
import paged_ref as ref
from test_paged_fp8_gpu import (DENSE, SCALES, SHARED, SPARSE, TILES, _all, _check_padding, _check_sparse, _dense, _sparse,  # noqa: F401
                                msa)
from test_paged_gpu import _dense as _dense16

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


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
def _check_eleven_bits(b, O, LSE, rows, heads):
    """ref8.check_attention's bounds, with P's own: fp16, 2^-11 of itself, or half of fp16's last step, 2^-25, in units that the
    largest P of a row's page was 2^7 in when they were set (128-row tiles; eight columns: 2^15). There V stands relative to
    its page's largest power of two 2^F, or, where a page's lie more than 2^14 apart, each vector to its own: for a token j
    that is 2^-32 max(p 2^F) |v_j| / 2^F_j."""
    import torch

    for r in rows:
        blocks = list(range(b.row_pos[r] // 128 + 1))
        at = b.table[b.row_seq[r], blocks].long()
        token = (torch.arange(len(blocks) * 128) <= b.row_pos[r])
        own_end = b.row_pos[r] + b.counts[b.row_seq[r]]  # (a page's powers of two are those of all rows' tokens)
        there = torch.arange(len(blocks) * 128).view(-1, 128) <= own_end
        for h in heads:
            g = h // b.hg
            o, lse, tol, tol_lse = ref.attend(b, r, h, blocks)
            k, v = (x[at, g].reshape(-1, 128)[token].double() for x in (b.K, b.V))
            f = b.V_exp[at, g].double() - 127
            largest = torch.where(there, f, -200.0).amax(1, keepdim=True).expand_as(f)
            least = torch.where(there & (f > -117), f, 200.0).amin(1, keepdim=True)
            unit = torch.where(largest - least > 14, f, largest).reshape(-1)[token]
            p = (k @ b.Q[r, h].double() / math.sqrt(128) - lse).exp()
            unit, top = torch.exp2(unit), float((p * torch.exp2(largest.reshape(-1)[token])).max())
            tol = tol + 2.0 ** -11 * (p @ v.abs()) + 2.0 ** -32 * top * (v.abs() / unit[:, None]).sum(0)
            err = (O[r, h].double() - o).abs()
            assert bool((err <= tol + 1e-30).all()), (r, h, float((err / (tol + 1e-30)).max()))
            assert abs(float(LSE[r, h]) - lse) <= tol_lse, (r, h)


def _some(b):
    return range(b.n) if b.n < 30 else range(0, b.n, 7), range(0, b.Hq, 1 if b.Hq <= 8 else 5)


@pytest.mark.parametrize("name", [*DENSE, *SCALES, *TILES, *SHARED])
def test_probabilities_have_eleven_bits(msa, name):  # noqa: F811
    """By eight columns, by 128-row tiles, behind a prefix that is shared or read as own pages."""
    b = ref8.Batch(seed=6, **{**DENSE, **SCALES, **TILES, **SHARED}[name])
    O, LSE = _dense(msa, b)
    _check_eleven_bits(b, O, LSE, *_some(b))
    _check_padding(b, O, LSE)


@pytest.mark.parametrize("what", ["spread", "spread a little", "pages", "rising pages", "falling pages", "zeros", "one large vector",
                                  "half a page large"])
@pytest.mark.parametrize("name", SCALES)
def test_eleven_bits_of_values_of_any_powers_of_two(msa, name, what):  # noqa: F811
    """V's powers of two differ from token to token and from page to page, by more and by less than fp16 holds."""
    import torch

    def change(b):
        gen = torch.Generator().manual_seed(5)
        some = lambda lo, hi, *shape: torch.exp2(torch.randint(lo, hi, shape, generator=gen).float())  # noqa: E731
        V = b.V.float()
        if what == "spread":
            V = V * some(-20, 20, *V.shape[:-1], 1)
        elif what == "spread a little":
            V = V * some(-6, 7, *V.shape[:-1], 1)
        elif what == "pages":
            V = V * some(-40, 40, V.shape[0], V.shape[1], 1, 1)
        elif what in ("rising pages", "falling pages"):
            for s in range(b.S):
                for c in range(b.prefix if s else 0, -(-b.lens[s] // 128)):
                    V[int(b.table[s, c])] *= 2.0 ** ((c * 3 if what[0] == "r" else -c * 3) % 90)
        elif what == "zeros":
            V[:, :, ::3] = torch.where(V[:, :, ::3].isnan(), NAN, 0.0)
        elif what == "one large vector":
            V[:, :, 17] *= 2.0 ** 40
        else:
            V[:, :, 64:] *= 2.0 ** 15
        b.V = V.to(torch.bfloat16)

    b = ref8.Batch(seed=9, change=change, **SCALES[name])
    O, LSE = _dense(msa, b)
    _check_eleven_bits(b, O, LSE, *_some(b))


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

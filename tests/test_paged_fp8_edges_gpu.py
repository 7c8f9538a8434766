"""Calls over a paged cache in 8 bits at the edges of what they take, on the GPU against their 64-bit forms (tests/paged_ref.py
and tests/paged_fp8_ref.py, bounds derived there)."""
import numpy as np
import pytest

import paged_fp8_ref as ref8
from test_paged_fp8_gpu import msa  # noqa: F401

pytestmark = pytest.mark.gpu


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

"""Plain 64-bit forms of the paged-cache operators and a builder of batches (test infrastructure).

Everything is row by row in numpy/torch float64, from the definitions in include/msa.h."""
import math

import numpy as np

BLOCK, D, E = 128, 128, 64


class Batch:
    """Random pools and a batch description. `counts` and `lens`: rows and lengths (new rows included) per sequence.
    Pages are drawn without order from a pool with `spare` unused ones; the slots behind a sequence's end, the unused
    pages and the page-table columns past the end hold `stale` (NaN, infinities, ...) and -1."""

    def __init__(self, counts, lens, Hq, G, pad=0, prefix=0, seed=0, spare=3, stale=float("nan"), max_blocks=None,
                 index=True, device="cuda"):
        import torch

        gen = torch.Generator().manual_seed(seed)
        self.S, self.Hq, self.G, self.hg, self.prefix = len(counts), Hq, G, Hq // G, prefix
        self.counts, self.lens = list(counts), list(lens)
        self.starts = [0]
        for c in counts:
            self.starts.append(self.starts[-1] + c)
        self.n = self.starts[-1]
        self.N = max(1, self.n + pad)
        blocks = [-(-x // BLOCK) for x in lens]
        self.max_blocks = max_blocks or max(max(blocks), prefix + 1)
        own = [max(0, b - prefix) for b in blocks]
        self.num_pages = prefix + sum(own) + spare
        order = torch.randperm(self.num_pages, generator=gen).to(torch.int32)
        table = torch.full((self.S, self.max_blocks), -1, dtype=torch.int32)
        at = prefix
        for i, b in enumerate(blocks):
            if counts[i]:
                table[i, :prefix] = order[:prefix]
            table[i, prefix:max(b, prefix)] = order[at:at + own[i]]
            at += own[i]

        def normal(*shape):
            return torch.randn(*shape, generator=gen).to(torch.bfloat16)

        self.K, self.V = normal(self.num_pages, G, BLOCK, D), normal(self.num_pages, G, BLOCK, D)
        self.k_idx = (normal(self.num_pages, BLOCK, E).float() + 0.5 * normal(self.num_pages, 1, E).float()).to(
            torch.bfloat16) if index else None
        for p in order[at:].tolist():
            self._fill(p, 0, stale)
        for i, (x, b) in enumerate(zip(lens, blocks)):
            if x % BLOCK and b > prefix:
                self._fill(int(table[i, b - 1]), x % BLOCK, stale)
        self.Q, self.q_idx = normal(self.N, Hq, D), normal(self.N, G, E)
        self.Q[self.n:] = stale
        self.q_idx[self.n:] = stale
        self.table = table
        self.row_seq = [i for i, c in enumerate(counts) for _ in range(c)]
        self.row_pos = [x - c + j for c, x in zip(counts, lens) for j in range(c)]
        self.device = device

    def _fill(self, page, slot, v):
        self.K[page, :, slot:] = v
        self.V[page, :, slot:] = v
        if self.k_idx is not None:
            self.k_idx[page, slot:] = v

    def gpu(self, k=16):
        """(shape, cache, dict of GPU tensors)"""
        import torch

        import block_sparse_attention_scores_gb300 as msa

        t = {n: getattr(self, n).cuda() for n in ("K", "V", "Q", "q_idx", "table")}
        t["k_idx"] = None if self.k_idx is None else self.k_idx.cuda()
        t["row_start"] = torch.tensor(self.starts, dtype=torch.int32, device="cuda")
        t["seq_len"] = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        shape = msa.PagedShape(S=self.S, N=self.N, Hq=self.Hq, G=self.G, num_pages=self.num_pages,
                               max_blocks=self.max_blocks, k=k, prefix_blocks=self.prefix)
        cache = msa.PagedCache(t["K"], t["V"], t["k_idx"], t["table"], t["row_start"], t["seq_len"])
        return shape, cache, t


def select(b, r, k):
    """block ids [G, k] of row r by exact scores (64-bit sums of exact products)."""
    seq, last = b.row_seq[r], b.row_pos[r] // BLOCK
    out = np.full((b.G, k), -1, np.int32)
    keys = b.k_idx[b.table[seq, :last].long()].double()  # [last, 128, E]
    for g in range(b.G):
        s = (keys @ b.q_idx[r, g].double()).nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf)
        pool = s.amax(1).tolist() if last else []
        ids = sorted(sorted(range(last), key=lambda c: (-pool[c], c))[:k - 1] + [last])
        out[g, :len(ids)] = ids
    return out


def attend(b, r, h, blocks, bf16_p=False):
    """O [D], LSE of head h of row r over the tokens <= its position of `blocks`, and bounds on what a kernel with bf16
    inputs, fp32 sums and a bf16 result may be off:

    * a score is a sum of 128 products in fp32: off by 128 * 2^-24 * sum |q k| scale at most, =: d; a probability by
      the factor e^(2 d) (its own score's error and the sum's), so O by 2 d sum p |v|, LSE by d;
    * exp2 in hardware, and the other fp32 operations of a term (a scaling, a rescaling, a product, a join): 2^-19 of
      sum p |v|; the sum's own additions stay below n 2^-24 of it, for n <= 2^13 tokens at a time 2^-11 at worst, in
      practice (errors of random sign, 128 partial sums) under 2^-19 as well;
    * probabilities kept as bf16 (`bf16_p`): 2^-8 of sum p |v|; as the sum of two: 2^-16 of it;
    * the result's own rounding: 2^-8 |O|."""
    import torch

    seq, t, g = b.row_seq[r], b.row_pos[r], h // b.hg
    blocks = [c for c in blocks if c >= 0]
    if not blocks:
        return torch.zeros(D, dtype=torch.float64), -math.inf, torch.zeros(D, dtype=torch.float64), 0.0
    at = b.table[seq, blocks].long()
    token = (torch.tensor(blocks)[:, None] * BLOCK + torch.arange(BLOCK)).reshape(-1)
    k = b.K[at, g].reshape(-1, D)[token <= t].double()
    v = b.V[at, g].reshape(-1, D)[token <= t].double()
    q = b.Q[r, h].double()
    s = k @ q / math.sqrt(D)
    lse = torch.logsumexp(s, 0)
    p = (s - lse).exp()
    o = p @ v
    d = float((k.abs() @ q.abs()).max()) / math.sqrt(D) * 128 * 2.0 ** -24
    mass = p @ v.abs()
    tol = 2.0 ** -8 * o.abs() + (2 * d + 2.0 ** -18 + (2.0 ** -8 if bf16_p else 2.0 ** -16)) * mass
    return o, float(lse), tol, d + 2.0 ** -18 * (1 + abs(float(lse)))


def check_attention(b, rows, heads, O, LSE, blocks_of, bf16_p=False):
    """O and LSE (CPU tensors) of these rows and heads against attend()."""
    for r in rows:
        for h in heads:
            o, lse, tol, tol_lse = attend(b, r, h, blocks_of(r, h // b.hg), bf16_p)
            err = (O[r, h].double() - o).abs()
            assert bool((err <= tol + 1e-30).all()), (
                f"row {r} (position {b.row_pos[r]}) head {h}: O off by {float((err / (tol + 1e-30)).max()):.2f} of what "
                f"it may be")
            got = float(LSE[r, h])
            assert got == lse or abs(got - lse) <= tol_lse, f"row {r} head {h}: LSE {got} against {lse}, {tol_lse:.2e}"


def rotated(x, pos, freq, interleaved):
    """x [..., dim] float64 of one row, turned as complex numbers; and |a| + |b| of each value's pair."""
    import torch

    m = freq.numel()
    y, mag = x.clone(), torch.zeros_like(x)
    if m:
        i = torch.arange(m)
        a, c = (2 * i, 2 * i + 1) if interleaved else (i, i + m)
        phase = pos * freq.double()
        z = torch.complex(x[..., a], x[..., c]) * torch.polar(torch.ones_like(phase), phase)
        y[..., a], y[..., c] = z.real, z.imag
        mag[..., a] = mag[..., c] = x[..., a].abs() + x[..., c].abs()
    return y, mag
